"""The bias's gradient does not hang on which other gradients are asked for: one order of summation, bit for bit."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import fp8
from test_gpu_fp8 import DEV, f64, randn, spread, within

pytestmark = pytest.mark.gpu


def cancelling(rows, N):
    """Columns whose large terms cancel: what is left shows the order in which they were added up."""
    a = spread(rows, N, 3)
    half = rows // 2
    a[half:2 * half] = -a[:half][torch.randperm(half, generator=torch.Generator().manual_seed(4))]
    a[0] = randn((N,), 5, 2.0**-8)
    return a


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (15, 144, 272), (70, 272, 176), (1003, 144, 2064), (5000, 272, 1296),
                                      (8192, 128, 4096), (3000, 64, 144), (20000, 16, 16)])
def test_bias_gradient_alone(rows, K, N):
    x8, w8 = dg.fp8_quantize(randn((rows, K), 1).to(DEV)), dg.fp8_quantize(randn((N, K), 2, K**-0.5).to(DEV), 128)
    dy = cancelling(rows, N)
    every = dg.fp8_linear_backward(x8, w8, dy.to(DEV), need_db=True)["bias"]
    err = rows * fp8.UP * f64(dy.abs()).sum(0)
    db = f64(dy).sum(0)
    within(every, (db, err + fp8.BF16 * (abs(db) + err)), "bias")
    for x, w, need in ((None, w8, (False, False, True)), (x8, None, (False, True, True)), (None, w8, (True, False, True)),
                       (x8, None, (False, False, True))):
        assert torch.equal(dg.fp8_linear_backward(x, w, dy.to(DEV), *need)["bias"], every), need


def test_bias_gradient_of_what_is_not_finite():
    w8, dy = dg.fp8_quantize(randn((144, 32), 2).to(DEV), 128), randn((300, 144), 3)
    dy[7, 5], dy[100, 130], dy[200, 130] = float("nan"), float("inf"), float("inf")
    g = [dg.fp8_linear_backward(None, w8, dy.to(DEV), dx, False, True)["bias"] for dx in (False, True)]
    for db in g:
        assert db[5].isnan() and db[130] == float("inf") and db.isfinite().sum() == 142
    ok = g[0].isfinite()
    assert torch.equal(g[0][ok], g[1][ok])

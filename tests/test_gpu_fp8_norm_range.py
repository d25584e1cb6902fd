"""The root-mean-square norm where squares, or their mean and eps together, leave binary32: every form of its kernels
(a warp a row, a CTA a row, the backward in two passes), bf16 and 8-bit results, gradients; eps up to what is accepted."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import fp8
from test_gpu_fp8 import DEV, f64, randn, u8, within

pytestmark = pytest.mark.gpu


def check(x, w, dy, dh, eps):
    """Forward in both forms and backward of rows x against binary64, with the bounds of ordinary rows."""
    eps = float(np.float32(eps))
    d = x.shape[1]
    ref = fp8.rms_norm(f64(x), f64(w), eps)
    within(dg.rms_norm(x.to(DEV), w.to(DEV), eps=eps), (ref, fp8.rms_norm_bound(ref)), "y")
    g = dg.rms_norm_backward(x.to(DEV), w.to(DEV), dy.to(DEV), None if dh is None else dh.to(DEV), eps=eps)
    refs = fp8.rms_norm_backward(f64(x), f64(w), f64(dy), None if dh is None else f64(dh), eps)
    within(g["x"], refs["x"], "dx")
    within(g["weight"], refs["weight"], "dw")
    if d % 16:
        return
    codes, scales = dg.rms_norm(x.to(DEV), w.to(DEV), eps=eps, fp8=True)
    got = u8(scales)
    lo, hi = (fp8.quantize(ref * (1 + s * fp8.NORM_REL))[1] for s in (-1, 1))
    assert np.all((got == lo) | (got == hi))
    step = np.repeat(fp8.scale_values(got), 128, axis=1)[:, :d] * 2.0**-10   # half of the smallest
    assert np.all(np.abs(fp8.values(u8(codes), got) - ref) <= np.maximum(2.0**-4 * np.abs(ref), step)
                  + 2 * fp8.NORM_REL * np.abs(ref))


WIDTHS = [8, 256, 512, 1288, 2048, 8192, 16400]


def rows(d, *exponents):
    x = randn((len(exponents), d), d)
    return (x.double() * 2.0 ** torch.tensor(exponents).double()[:, None]).to(x.dtype)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("upstream", [False, True])
def test_rows_whose_squares_overflow(d, upstream):
    x = rows(d, 0, 100, -100, 64, 120, 3)
    w, dy = randn((d,), 2), randn((6, d), 3)
    check(x, w, dy, randn((6, d), 4) if upstream else None, 1e-6)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("eps", [1e30, 1e36, 3.3e38])
def test_large_eps(d, eps):
    """Rows below, beside and above eps; its sum with their mean square goes past binary32 for some."""
    x = rows(d, 0, 50, 60, 62, 63, 64, 70)
    check(x, randn((d,), 2), randn((7, d), 3), None, eps)

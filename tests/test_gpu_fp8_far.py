"""Block-scaled e4m3 operators on tensors whose offsets pass 2^31 elements or 2^32 bytes."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import fp8
from test_gpu_fp8 import BF16, DEV, f64, u8, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device=DEV).normal_(0, scale, generator=g)


def values(pair, part, block_rows=1):
    return fp8.values(u8(pair[0][part]), u8(pair[1][part]), block_rows)


def test_quantize_and_linear_of_many_rows():
    rows, K, N = 524500, 4112, 256                   # 2^31 values at row 522254
    x, w = normal((rows, K), 1), normal((N, K), 2, K**-0.5)
    x8, w8 = dg.fp8_quantize(x), dg.fp8_quantize(w, 128)
    back, y = dg.fp8_dequantize(*x8), dg.fp8_linear(x8, w8)
    wv = fp8.values(u8(w8[0]), u8(w8[1]), 128)
    for r in (0, 261100, 522252, rows - 3):
        part = slice(r, r + 3)
        q, s = fp8.quantize(f64(x[part]))
        assert np.array_equal(u8(x8[0][part]), q) and np.array_equal(u8(x8[1][part]), s)
        assert np.array_equal(f64(back[part]), fp8.values(q, s))
        within(y[part], fp8.linear(fp8.values(q, s), wv), f"rows {r}")


@pytest.mark.parametrize("rows", [2, 300])
def test_linear_with_a_large_weight(rows):
    N, K = 70016, 32768                              # 2^31 codes at row 65536
    w8 = dg.fp8_quantize(normal((N, K), 3, K**-0.5), 128)
    x = normal((rows, K), 4)
    x8 = dg.fp8_quantize(x)
    y = dg.fp8_linear(x8, w8)
    xv = values(x8, slice(0, 2))
    for n in (0, 65536, 69888):
        part, blocks = slice(n, n + 128), slice(n // 128, n // 128 + 1)
        wv = fp8.values(u8(w8[0][part]), u8(w8[1][blocks]), 128)
        within(y[:2, part], fp8.linear(xv, wv), f"features {n}")


def test_backward_of_many_rows():
    rows, K, N = 530000, 256, 4112                   # dy passes 2^31 values
    x8, w8 = dg.fp8_quantize(normal((rows, K), 5)), dg.fp8_quantize(normal((N, K), 6, K**-0.5), 128)
    dy = torch.zeros((rows, N), dtype=BF16, device=DEV)
    picked = [0, 1, 261000, 522300, rows - 1]        # the rows whose gradient is not zero
    dy[picked] = normal((len(picked), N), 7)
    g = dg.fp8_linear_backward(x8, w8, dy, need_db=True)
    wv = fp8.values(u8(w8[0]), u8(w8[1]), 128)
    xv = np.concatenate([values(x8, slice(r, r + 1)) for r in picked])
    ref = fp8.linear_backward(xv, wv, f64(dy[picked]))
    for n in ("x", "weight", "bias"):
        within(g[n][picked] if n == "x" else g[n], ref[n], n)
    assert not g["x"][2:260000].any()


@pytest.mark.parametrize("rows,d", [(70000, 32768), (530000, 4104)])
def test_norm_of_many_rows(rows, d):
    x, w = normal((rows, d), 8), normal((d,), 9)
    y = dg.rms_norm(x, w)
    picked = [0, 32767, 65537, rows - 1]
    ref = fp8.rms_norm(f64(x[picked]), f64(w), 1e-6)
    within(y[picked], (ref, fp8.rms_norm_bound(ref)), "y")
    del y
    dy = torch.zeros((rows, d), dtype=BF16, device=DEV)
    dy[picked] = normal((len(picked), d), 10)
    g = dg.rms_norm_backward(x, w, dy)
    refs = fp8.rms_norm_backward(f64(x[picked]), f64(w), f64(dy[picked]), None, 1e-6)
    within(g["x"][picked], refs["x"], "x")
    within(g["weight"], refs["weight"], "weight")
    if d % 16 == 0:
        codes, scales = dg.rms_norm(x, w, fp8=True)
        v = np.concatenate([values((codes, scales), slice(r, r + 1)) for r in picked])
        assert np.all(np.abs(v - ref) <= 2.0**-4 * np.abs(ref) * (1 + 2**-10) + 2.0**-10 * np.abs(ref).max())

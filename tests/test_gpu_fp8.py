"""Block-scaled e4m3 operators against the fp64 reference.

Codes, scales and everything read back are compared bit for bit; sums and norms
per element with the bounds that oracle/fp8.py derives (binary32 sums of n terms:
n * 2^-23 of the sum of magnitudes; a rounding to bf16: 2^-8 of the value)."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import fp8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16, E4M3, E8M0 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def f64(t):
    return t.detach().cpu().double().numpy()


def u8(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16)


def within(got, ref, what):
    (ref, bound), got = ref, f64(got)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(got - ref)):.3e}, {np.max(over):.3e} over the bound"


def spread(rows, K, seed):
    """Rows of many magnitudes, so that neighbouring blocks have far scales."""
    x = randn((rows, K), seed)
    x *= (2.0 ** torch.randint(-6, 7, (rows, 1), generator=torch.Generator().manual_seed(seed + 1))).to(BF16)
    return x


def held(x, block_rows=1):
    """(pair on the GPU, its values in binary64) of a bf16 tensor."""
    codes, scales = fp8.quantize(f64(x), block_rows)
    pair = torch.from_numpy(codes).view(E4M3).to(DEV), torch.from_numpy(scales).view(E8M0).to(DEV)
    return pair, fp8.values(codes, scales, block_rows)


# ------------------------------------------------------------------ the format

def odd_values(rows, K, seed):
    """Blocks that go wrong: zeros, subnormals, an amax on the border of a scale, huge, NaN, infinity."""
    x = randn((rows, K), seed)
    x *= (2.0 ** torch.randint(-30, 30, (rows, 1), generator=torch.Generator().manual_seed(seed + 1))).to(BF16)
    f = x.view(-1)
    for i, v in enumerate((0.0, 1e-40, 448.0, 450.0, 2.0**-133, 3.3e38, 2.0**-125)):
        if f.numel() >= 128 * (i + 2):
            f[128 * i:128 * i + 128] = v
            f[128 * i + 5] = -v / 2
    if f.numel() >= 2048:
        f[1300], f[1500] = float("nan"), float("-inf")
    return x


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 112), (1, 128), (7, 144), (128, 128), (129, 272), (300, 1296), (257, 2048),
                                    (5, 4096)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_bit_exact(rows, K, block_rows):
    x = odd_values(rows, K, rows + K)
    codes, scales = dg.fp8_quantize(x.to(DEV), block_rows)
    q, s = fp8.quantize(f64(x), block_rows)
    assert np.array_equal(u8(scales), s)
    assert np.array_equal(u8(codes) & 0x7F, q & 0x7F) and np.array_equal(u8(codes)[q & 0x7F != 0x7F], q[q & 0x7F != 0x7F])
    back = f64(dg.fp8_dequantize(codes, scales))
    # magnitudes over 31/32 of 2^128 round to 2^128, an infinity in bf16; every other value is a bf16 number
    v = fp8.values(q, s, block_rows)
    assert np.array_equal(back, np.where(np.abs(v) == 2.0**128, np.copysign(np.inf, v), v), equal_nan=True)


def test_quantize_leading_dimensions_and_empty():
    x = randn((3, 5, 272), 2)
    codes, scales = dg.fp8_quantize(x.to(DEV))
    assert codes.shape == x.shape and scales.shape == (3, 5, 3)
    q, s = fp8.quantize(f64(x).reshape(15, 272))
    assert np.array_equal(u8(codes).reshape(15, 272), q) and np.array_equal(u8(scales).reshape(15, 3), s)
    assert np.array_equal(f64(dg.fp8_dequantize(codes, scales)).reshape(15, 272), fp8.values(q, s))
    for block_rows in (1, 128):
        codes, scales = dg.fp8_quantize(torch.empty((0, 64), dtype=BF16, device=DEV), block_rows)
        assert codes.shape == (0, 64) and scales.shape == (0, 1) and dg.fp8_dequantize(codes, scales).shape == (0, 64)


def test_dequantize_every_scale():
    """All 256 scale bytes and all codes, also those that the quantiser does not write."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(2).view(256, 2).contiguous()
    got = f64(dg.fp8_dequantize(codes.view(E4M3).to(DEV), scales.view(E8M0).to(DEV)))
    with np.errstate(over="ignore"):
        ref = fp8.bf16_rne(fp8.values(codes.numpy(), scales.numpy()).astype(np.float32))
    assert np.array_equal(got, ref, equal_nan=True)


# ------------------------------------------------------------------ linear

LINEAR = [(1, 16, 16), (1, 4096, 256), (2, 128, 240), (7, 144, 224), (16, 512, 448), (17, 528, 464), (33, 2064, 128),
          (64, 1024, 1024), (100, 1296, 2064), (128, 640, 272), (129, 256, 512), (256, 896, 224), (257, 384, 688),
          (511, 2048, 480), (1000, 272, 1296), (3, 8192, 144), (40, 8208, 272), (65, 4112, 128), (100, 8192, 528),
          (128, 8208, 400), (300, 12288, 272), (260, 400, 7168), (1300, 272, 4112)]


@pytest.mark.parametrize("rows,K,N", LINEAR)
@pytest.mark.parametrize("bias", [False, True])
def test_linear(rows, K, N, bias):
    (x8, x), (w8, w) = held(spread(rows, K, rows)), held(randn((N, K), N, K**-0.5), 128)
    b = randn((N,), 5) if bias else None
    y = dg.fp8_linear(x8, w8, None if b is None else b.to(DEV))
    within(y, fp8.linear(x, w, None if b is None else f64(b)), "y")


@pytest.mark.parametrize("rows,K,N", [(3, 2176, 400), (40, 1152, 656), (300, 1664, 528), (7, 8320, 144), (90, 8320, 400)])
def test_every_block_has_its_own_scale(rows, K, N):
    """Codes of one, scales of all sizes: each sum is that of its own blocks' scales, exactly."""
    rng = np.random.default_rng(rows)
    kb, nb = -(-K // 128), -(-N // 128)
    xs = rng.integers(127 - 4, 127 + 5, (rows, kb)).astype(np.uint8)
    ws = rng.integers(127 - 4, 127 + 5, (nb, kb)).astype(np.uint8)
    one = lambda shape: torch.full(shape, 0x38, dtype=torch.uint8, device=DEV).view(E4M3)
    x, w = np.full((rows, K), 0x38, np.uint8), np.full((N, K), 0x38, np.uint8)
    y = dg.fp8_linear((one((rows, K)), torch.from_numpy(xs).view(E8M0).to(DEV)),
                      (one((N, K)), torch.from_numpy(ws).view(E8M0).to(DEV)))
    exact = fp8.values(x, xs) @ fp8.values(w, ws, 128).T   # multiples of 2^-8 below 2^16: 24 bits
    assert np.array_equal(f64(y), fp8.bf16_rne(exact.astype(np.float32)))


def test_linear_from_bf16_and_leading_dimensions():
    x = randn((2, 3, 272), 1)
    w8, w = held(randn((160, 272), 2), 128)
    y = dg.fp8_linear(x.to(DEV), w8)
    assert y.shape == (2, 3, 160)
    ref = fp8.linear(held(x.view(6, 272))[1], w)
    within(y.view(6, 160), ref, "y")
    out = torch.empty_like(y)
    assert dg.fp8_linear(dg.fp8_quantize(x.to(DEV)), w8, out=out) is out and torch.equal(out, y)
    assert dg.fp8_linear(x.to(DEV)[:0], w8).shape == (0, 3, 160)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 17, 200])
@pytest.mark.parametrize("K,N", [(16, 16), (144, 240), (640, 400), (2064, 272), (8208, 144)])
def test_bf16_rows_give_what_their_codes_give(rows, K, N):
    """Up to four rows the product quantises x itself: the same codes, the same sums."""
    x = odd_values(rows, K, rows + K)
    w8, b = dg.fp8_quantize(randn((N, K), 2, K**-0.5).to(DEV), 128), randn((N,), 3).to(DEV)
    y = dg.fp8_linear(x.to(DEV), w8, b)
    assert torch.equal(y.view(torch.int16), dg.fp8_linear(dg.fp8_quantize(x.to(DEV)), w8, b).view(torch.int16)) or \
        torch.equal(torch.nan_to_num(y, 7.0), torch.nan_to_num(dg.fp8_linear(dg.fp8_quantize(x.to(DEV)), w8, b), 7.0))


@pytest.mark.parametrize("K", [272, 2048])
def test_parts_of_the_rows(K):
    """Activations sliced by rows: their scales begin at any byte."""
    x, w8, dy = randn((300, K), 1).to(DEV), dg.fp8_quantize(randn((160, K), 2).to(DEV), 128), randn((300, 160), 3).to(DEV)
    codes, scales = dg.fp8_quantize(x)
    xv, wv = fp8.values(u8(codes), u8(scales)), fp8.values(u8(w8[0]), u8(w8[1]), 128)
    for a, b in ((3, 20), (7, 300), (299, 300)):
        part = codes[a:b], scales[a:b]
        assert torch.equal(dg.fp8_linear(part, w8), dg.fp8_linear(tuple(t.clone() for t in part), w8))
        within(dg.fp8_linear(part, w8), fp8.linear(xv[a:b], wv), "rows of y")
        assert torch.equal(dg.fp8_dequantize(*part), dg.fp8_dequantize(codes, scales)[a:b])
        assert torch.equal(dg.fp8_linear_backward(part, w8, dy[a:b])["weight"],
                           dg.fp8_linear_backward(tuple(t.clone() for t in part), w8, dy[a:b])["weight"])


@pytest.mark.parametrize("rows", [1, 5, 40, 200])
def test_what_is_not_finite_stays_in_its_row(rows):
    x, w = randn((rows, 512), 1), randn((288, 512), 2)
    clean = dg.fp8_linear(x.to(DEV), dg.fp8_quantize(w.to(DEV), 128))
    x[rows // 2, 300] = float("inf")
    w[7, 130] = float("nan")
    got = dg.fp8_linear(x.to(DEV), dg.fp8_quantize(w.to(DEV), 128)).cpu()
    bad = torch.zeros(rows, 288, dtype=torch.bool)
    bad[rows // 2], bad[:, :128] = True, True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean.cpu()[~bad])


def test_tiny_and_huge_scales():
    """Sums near both ends of bf16's range."""
    for ex, ew in ((-60, -60), (60, 60), (-110, 100), (-124, 7)):
        x = randn((9, 256), 1).double() * 2.0**ex
        w = randn((64, 256), 2).double() * 2.0**ew
        (x8, xv), (w8, wv) = held(x.to(BF16)), held(w.to(BF16), 128)
        within(dg.fp8_linear(x8, w8), fp8.linear(xv, wv), (ex, ew))


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (2, 128, 240), (17, 528, 464), (100, 1296, 2064), (129, 256, 512),
                                      (257, 384, 688), (1000, 272, 1296), (640, 2048, 224), (2048, 144, 272), (2100, 528, 400)])
def test_linear_backward(rows, K, N):
    (x8, x), (w8, w) = held(spread(rows, K, rows)), held(randn((N, K), N, K**-0.5), 128)
    dy = spread(rows, N, 9)
    g = dg.fp8_linear_backward(x8, w8, dy.to(DEV), need_db=True)
    ref = fp8.linear_backward(x, w, f64(dy))
    for n in ("x", "weight", "bias"):
        within(g[n], ref[n], n)
    only = dg.fp8_linear_backward(None, w8, dy.to(DEV), need_dw=False)
    assert torch.equal(only["x"], g["x"]) and only["weight"] is None and only["bias"] is None
    only = dg.fp8_linear_backward(x8, None, dy.to(DEV), need_dx=False)
    assert torch.equal(only["weight"], g["weight"]) and only["x"] is None


def test_linear_backward_of_no_rows():
    (x8, _), (w8, _) = held(randn((1, 64), 1)), held(randn((32, 64), 2), 128)
    x8 = tuple(t[:0] for t in x8)
    g = dg.fp8_linear_backward(x8, w8, torch.empty((0, 32), dtype=BF16, device=DEV), need_db=True)
    assert g["x"].shape == (0, 64) and not g["weight"].any() and not g["bias"].any()


# ------------------------------------------------------------------ norm

NORM = [(1, 8), (3, 120), (9, 128), (2, 136), (5, 256), (33, 264), (7, 1024), (100, 1288), (1000, 2048), (3, 2056),
        (600, 4096), (4, 5120), (3, 8192), (2, 16384), (2, 16400), (3, 32768)]


@pytest.mark.parametrize("rows,d", NORM)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_gradients(rows, d, residual):
    x, w, dy = spread(rows, d, rows + d), randn((d,), 1), randn((rows, d), 3)
    r, dh = (randn((rows, d), 2), randn((rows, d), 4)) if residual else (None, None)
    to = lambda t: None if t is None else t.to(DEV)
    out = dg.rms_norm(to(x), to(w), to(r), eps=1e-5)
    y, h = out if residual else (out, to(x))
    hv = fp8.add(f64(x), f64(r)) if residual else f64(x)
    assert np.array_equal(f64(h), hv)
    ref = fp8.rms_norm(hv, f64(w), 1e-5)
    within(y, (ref, fp8.rms_norm_bound(ref)), "y")
    g = dg.rms_norm_backward(h, to(w), to(dy), to(dh), eps=1e-5)
    refs = fp8.rms_norm_backward(hv, f64(w), f64(dy), None if dh is None else f64(dh), 1e-5)
    within(g["x"], refs["x"], "dx")
    within(g["weight"], refs["weight"], "dw")
    again = dg.rms_norm_backward(h, to(w), to(dy), to(dh), eps=1e-5)
    assert torch.equal(again["weight"], g["weight"])
    assert torch.equal(dg.rms_norm_backward(h, to(w), to(dy), to(dh), eps=1e-5, need_dw=False)["x"], g["x"])
    assert torch.equal(dg.rms_norm_backward(h, to(w), to(dy), to(dh), eps=1e-5, need_dx=False)["weight"], g["weight"])


@pytest.mark.parametrize("rows,d", [(1, 16), (3, 112), (9, 128), (5, 272), (100, 1296), (1000, 2048), (600, 4096), (3, 8192),
                                    (2, 16400), (2, 32768)])
def test_norm_in_8_bits(rows, d):
    """Scales and codes are those of the exact values but where these lie within the norm's own error of a border."""
    x, w, r = spread(rows, d, rows + d), randn((d,), 1), randn((rows, d), 2)
    (codes, scales), h = dg.rms_norm(x.to(DEV), w.to(DEV), r.to(DEV), eps=1e-5, fp8=True)
    y = fp8.rms_norm(fp8.add(f64(x), f64(r)), f64(w), 1e-5)
    assert np.array_equal(f64(h), fp8.add(f64(x), f64(r)))
    got = u8(scales)
    lo = fp8.quantize(y * (1 - fp8.NORM_REL))[1]
    hi = fp8.quantize(y * (1 + fp8.NORM_REL))[1]
    assert np.all((got == lo) | (got == hi))
    v = fp8.values(u8(codes), got)
    step = np.repeat(fp8.scale_values(got), 128, axis=1)[:, :d] * 2.0**-10   # half of the smallest
    assert np.all(np.abs(v - y) <= np.maximum(2.0**-4 * np.abs(y), step) + 2 * fp8.NORM_REL * np.abs(y))
    plain = dg.rms_norm(x.to(DEV), w.to(DEV), r.to(DEV), eps=1e-5)[0]
    assert np.all(np.abs(f64(plain) - v) <= np.maximum(2.0**-4 * np.abs(y), step) + 2.0**-7 * np.abs(y))


def test_norm_rows_of_zeros_and_of_large_values():
    x = randn((6, 512), 1)
    x[1] = 0
    x[2] *= 2.0**100      # squares beyond binary32
    x[3] *= 2.0**-100
    x[4, 9] = float("nan")
    w, dy = randn((512,), 2), randn((6, 512), 3)
    ok = [0, 1, 2, 3, 5]
    ref = fp8.rms_norm(f64(x), f64(w), 1e-6)
    y = dg.rms_norm(x.to(DEV), w.to(DEV))
    assert torch.isnan(y[4]).all()
    within(y[ok], (ref[ok], fp8.rms_norm_bound(ref[ok])), "y")
    codes, scales = dg.rms_norm(x.to(DEV), w.to(DEV), fp8=True)
    assert (u8(scales)[4] == 255).all() and not (u8(codes)[1] & 0x7F).any() and (u8(scales)[1] == 127).all()
    g = dg.rms_norm_backward(x[ok].to(DEV), w.to(DEV), dy[ok].to(DEV))
    refs = fp8.rms_norm_backward(f64(x[ok]), f64(w), f64(dy[ok]), None, 1e-6)
    within(g["x"], refs["x"], "dx")
    within(g["weight"], refs["weight"], "dw")
    g = dg.rms_norm_backward(x.to(DEV)[:0], w.to(DEV), dy.to(DEV)[:0])
    assert g["x"].shape == (0, 512) and not g["weight"].any()


# ------------------------------------------------------------------ layers

def leaf(t):
    return t.to(DEV).requires_grad_()


@pytest.mark.parametrize("bias", [False, True])
def test_linear_layer(bias):
    x, w, b, dy = leaf(randn((3, 50, 272), 1)), leaf(randn((304, 272), 2, 0.06)), leaf(randn((304,), 3)), randn((3, 50, 304), 4)
    y = dg.fp8_linear_layer(x, w, b if bias else None)
    xv, wv = held(x.detach().view(150, 272).cpu())[1], held(w.detach().cpu(), 128)[1]
    within(y.view(150, 304), fp8.linear(xv, wv, f64(b) if bias else None), "y")
    y.backward(dy.to(DEV))
    ref = fp8.linear_backward(xv, wv, f64(dy).reshape(150, 304))
    within(x.grad.view(150, 272), ref["x"], "x")
    within(w.grad, ref["weight"], "weight")
    if bias:
        within(b.grad, ref["bias"], "bias")
    # only what is asked for, and a gradient that arrives broadcast
    (gw,) = torch.autograd.grad(dg.fp8_linear_layer(x.detach(), w).sum(), (w,))
    ones = np.ones((150, 304))
    within(gw, fp8.linear_backward(xv, wv, ones)["weight"], "weight of a sum")


@pytest.mark.parametrize("residual", [False, True])
def test_norm_layer(residual):
    x, w, r = leaf(randn((2, 20, 136), 1)), leaf(randn((136,), 2)), leaf(randn((2, 20, 136), 3))
    dy, dh = randn((40, 136), 4), randn((40, 136), 5)
    out = dg.rms_norm_layer(x, w, r if residual else None)
    hv = fp8.add(f64(x), f64(r)) if residual else f64(x)
    hv = hv.reshape(40, 136)
    up = [dy.view(2, 20, 136).to(DEV), dh.view(2, 20, 136).to(DEV)]
    gx, gw, *gr = torch.autograd.grad(out, (x, w, r) if residual else (x, w), up if residual else up[:1])
    ref = fp8.rms_norm_backward(hv, f64(w), f64(dy), f64(dh) if residual else None, 1e-6)
    within(gx.view(40, 136), ref["x"], "x")
    within(gw, ref["weight"], "weight")
    if residual:
        assert torch.equal(gr[0], gx)
        # h alone is used: the norm passes its gradient on
        (gx,) = torch.autograd.grad(dg.rms_norm_layer(x, w, r)[1], (x,), up[1])
        assert torch.equal(gx, up[1])


@pytest.mark.parametrize("residual", [False, True])
def test_norm_linear_layer(residual):
    x, r = leaf(randn((60, 272), 1)), leaf(randn((60, 272), 2))
    nw, w, b = leaf(randn((272,), 3)), leaf(randn((320, 272), 4, 0.06)), leaf(randn((320,), 5))
    dy, dh = randn((60, 320), 6), randn((60, 272), 7)
    out = dg.fp8_norm_linear_layer(x, nw, w, b, r if residual else None, eps=1e-5)
    y, h = out if residual else (out, x)
    n8 = dg.rms_norm(x.detach(), nw.detach(), r.detach() if residual else None, eps=1e-5, fp8=True)
    n8 = n8[0] if residual else n8
    nv, wv = fp8.values(u8(n8[0]), u8(n8[1])), held(w.detach().cpu(), 128)[1]
    within(y, fp8.linear(nv, wv, f64(b)), "y")
    leaves = (x, nw, w, b) + ((r,) if residual else ())
    g = torch.autograd.grad(out, leaves, [dy.to(DEV), dh.to(DEV)][:1 + residual])
    ref = fp8.linear_backward(nv, wv, f64(dy))
    within(g[2], ref["weight"], "weight")
    within(g[3], ref["bias"], "bias")
    dn = dg.fp8_linear_backward(n8, dg.fp8_quantize(w.detach(), 128), dy.to(DEV), need_dw=False)["x"]
    within(dn, ref["x"], "the norm's result")
    refs = fp8.rms_norm_backward(f64(h), f64(nw), f64(dn), f64(dh) if residual else None, 1e-5)
    within(g[0], refs["x"], "x")
    within(g[1], refs["weight"], "norm weight")
    if residual:
        assert torch.equal(g[4], g[0])


def test_tp_layers_that_keep_8_bits():
    """The forward is the bf16 layer's bit for bit, the backward that of the values that the codes stand for."""
    x, w, b, dy = leaf(randn((2, 33, 144), 1)), leaf(randn((176, 144), 2, 0.1)), leaf(randn((176,), 3)), randn((2, 33, 176), 4).to(DEV)
    y = dg.tp_linear_layer_keep8(x, w, b)
    assert torch.equal(y, dg.tp_linear(x.detach(), w.detach(), b.detach()))
    g = torch.autograd.grad(y, (x, w, b), dy)
    xv = dg.fp8_dequantize(*dg.fp8_quantize(x.detach()))
    ref = dg.tp_linear_backward(xv, w.detach(), dy, need_db=True)
    assert all(torch.equal(a, ref[n]) for a, n in zip(g, ("x", "weight", "bias")))
    exact = f64(dy).reshape(66, 176).T @ held(x.detach().cpu().view(66, 144))[1]
    within(g[1], (exact, fp8.product_bound(f64(dy).reshape(66, 176).T, f64(xv).reshape(66, 144), exact)), "weight")

    x, w13, w2, dy = leaf(randn((2, 1, 16, 64), 5)), leaf(randn((2, 64, 64), 6, 0.2)), leaf(randn((64, 64), 7, 0.2)), randn((2, 1, 16, 64), 8).to(DEV)
    y = dg.tp_swiglu_layer_keep8(x, w13, w2)
    assert torch.equal(y, dg.tp_swiglu(x.detach(), w13.detach(), w2.detach()))
    g = torch.autograd.grad(y, (x, w13, w2), dy)
    ref = dg.tp_swiglu_backward(dg.fp8_dequantize(*dg.fp8_quantize(x.detach())), w13.detach(), w2.detach(), dy)
    assert all(torch.equal(a, ref[n]) for a, n in zip(g, ("x", "w13", "w2")))


@pytest.mark.parametrize("layer", ["fp8_linear_layer", "tp_linear_layer_keep8", "fp8_norm_linear_layer"])
def test_what_a_layer_keeps(layer):
    """Bytes held for the backward: one a value of the input (and one scale in 128), not two."""
    x, w = leaf(randn((512, 256), 1)), leaf(randn((128, 256), 2))
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t), t)[1], lambda t: t):
        if layer == "fp8_norm_linear_layer":
            dg.fp8_norm_linear_layer(x, leaf(randn((256,), 3)), w)
            kept = [t for t in kept if t.data_ptr() != x.data_ptr()]   # the residual stream itself
        else:
            getattr(dg, layer)(x, w)
    held_bytes = sum(t.numel() * t.element_size() for t in kept if t.shape[:1] == (512,))
    assert held_bytes == 512 * 256 + 512 * 2


def test_layers_refuse_a_second_derivative():
    x, w = leaf(randn((4, 32), 1)), leaf(randn((16, 32), 2))
    (g,) = torch.autograd.grad(dg.fp8_linear_layer(x, w).sum(), (x,), create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("layer", ["fp8_linear_layer", "tp_linear_layer_keep8", "fp8_norm_linear_layer"])
@pytest.mark.parametrize("trained", ["x", "w", "b", "xw", "xb", "wb"])
def test_layers_with_frozen_inputs(layer, trained):
    """The gradients that are asked for are bit for bit those of the layer with everything trained; of x nothing more
    than the layer's input is kept where the weight is frozen."""
    x, w, b, dy = randn((70, 272), 1), randn((176, 272), 2, 0.1), randn((176,), 3), randn((70, 176), 4).to(DEV)
    nw = randn((272,), 5).to(DEV)

    def grads(names):
        t = {n: v.to(DEV).requires_grad_(n in names) for n, v in (("x", x), ("w", w), ("b", b))}
        kept = []
        with torch.autograd.graph.saved_tensors_hooks(lambda v: (kept.append(v), v)[1], lambda v: v):
            if layer == "fp8_norm_linear_layer":
                y = dg.fp8_norm_linear_layer(t["x"], nw, t["w"], t["b"])
            else:
                y = getattr(dg, layer)(t["x"], t["w"], t["b"])
        if "w" not in names:
            assert not [v for v in kept if v.shape[:1] == (70,) and v.data_ptr() != t["x"].data_ptr()]
        return dict(zip(names, torch.autograd.grad(y, [t[n] for n in names], dy)))

    every, some = grads("xwb"), grads(trained)
    assert all(torch.equal(some[n], every[n]) for n in trained)

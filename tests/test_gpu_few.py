"""Few-token operators (4-bit weights, routed experts) against the fp64 oracle.

Tolerances are per element and derived from the arithmetic: products summed in
binary32 over n terms are off by at most n * 2^-23 * sum |w||x| (every partial
sum off by at most one unit), a result rounded to bf16 by 2^-8 of itself; the
routed layer's bound is written out in oracle/few.py.  Codes, scales, zero
points, choices and everything read back are compared bit for bit."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import few

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16)


def within(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(got - ref)):.3e}, {np.max(over):.3e} over the bound"


# ------------------------------------------------------------------ 4-bit weights

def odd_weights(rows, K, seed):
    """Weights of many magnitudes with the groups that go wrong: zeros, one value, subnormals, huge, one-sided."""
    w = randn((rows, K), seed)
    w *= (2.0 ** torch.randint(-20, 20, (rows, 1), generator=torch.Generator().manual_seed(seed + 1))).to(BF16)
    f = w.view(-1)
    f[:32] = 0
    if f.numel() >= 256:
        f[128:160] = f[128:160].abs()
        f[160:192] = -f[160:192].abs()
        f[192:224] = torch.tensor(3.0e38)
        f[224:256] = torch.tensor(1.0e-40)
    return w


@pytest.mark.parametrize("rows,K,group", [(1, 32, 32), (3, 64, 32), (17, 128, 64), (5, 256, 128), (130, 96, 32),
                                          (33, 1024, 128), (7, 4096, 64)])
@pytest.mark.parametrize("zero_points", [False, True])
def test_w4_quantize_bit_exact(rows, K, group, zero_points):
    w = odd_weights(rows, K, rows + K)
    codes, scales, zeros = dg.w4_quantize(w.to(DEV), group, zero_points=zero_points)
    q, s, z = few.w4_quantize(f64(w), group, zero_points)
    assert np.array_equal(f64(scales), s)
    assert np.array_equal(codes.cpu().numpy(), few.w4_pack(q))
    assert (zeros is None) == (not zero_points)
    if zero_points:
        assert np.array_equal(zeros.cpu().numpy(), z)
    back = dg.w4_dequantize(codes, scales, zeros)
    want = few.bf16_rne(few.w4_values(few.w4_pack(q), s, z if zero_points else None).astype(np.float32))
    assert np.array_equal(f64(back), want)


@pytest.mark.parametrize("zero_points", [False, True])
def test_w4_quantize_nonfinite_groups_are_nan(zero_points):
    w = randn((4, 128), 5)
    w[0, 3], w[1, 40], w[2, 64] = float("nan"), float("inf"), float("-inf")
    w[3, 96], w[3, 97] = 3.0e38, -3.0e38       # a range beyond binary32: no finite scale with zero points
    bad = 4 if zero_points else 3
    codes, scales, zeros = dg.w4_quantize(w.to(DEV), 32, zero_points=zero_points)
    q, s, z = few.w4_quantize(f64(w), 32, zero_points)
    assert np.array_equal(f64(scales), s, equal_nan=True) and np.isnan(s).sum() == bad
    assert np.array_equal(codes.cpu().numpy(), few.w4_pack(q))
    back = f64(dg.w4_dequantize(codes, scales, zeros))
    assert np.isnan(back[0, :32]).all() and np.isnan(back).sum() == 32 * bad


def test_w4_quantize_every_tie():
    # all bf16 significands against a group maximum of 7: every quotient that can fall on a half
    v = torch.arange(0, 7 * 256 + 1, dtype=torch.float32) / 256
    v = torch.cat([v, -v]).to(BF16)
    w = torch.zeros((-(-v.numel() // 31), 32), dtype=BF16)
    w[:, 0] = 7.0
    w[:, 1:].reshape(-1)
    flat = torch.zeros(w.shape[0] * 31, dtype=BF16)
    flat[: v.numel()] = v
    w[:, 1:] = flat.view(-1, 31)
    codes, scales, _ = dg.w4_quantize(w.to(DEV), 32)
    q, s, _ = few.w4_quantize(f64(w), 32, False)
    assert np.array_equal(codes.cpu().numpy(), few.w4_pack(q)) and np.array_equal(f64(scales), s)


def w4_weight(lead, N, K, group, zeros, seed):
    """Random codes over the whole range, scales near 1/sqrt(K): (device tensors, fp64 values)."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (*lead, N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand((*lead, N, K // group), generator=g) + 0.5) / (4 * K**0.5)).to(BF16)
    z = torch.randint(0, 16, (*lead, N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    values = few.w4_values(codes.numpy(), f64(scales), None if z is None else z.numpy())
    return tuple(None if t is None else t.to(DEV) for t in (codes, scales, z)), values


def w4_terms(w):
    """few.w4_magnitudes of a device weight."""
    return few.w4_magnitudes(w[0].cpu().numpy(), f64(w[1]), None if w[2] is None else w[2].cpu().numpy())


def check_linear(rows, K, N, group, zeros, bias, seed=0):
    x = randn((rows, K), seed + rows)
    w, values = w4_weight((), N, K, group, zeros, seed + K + N)
    b = randn((N,), seed + 9) if bias else None
    y = dg.w4_linear(x.to(DEV), *w, bias=None if b is None else b.to(DEV))
    ref = few.w4_linear(f64(x), values, None if b is None else f64(b))
    # sums of codes * x and of zero points * x, made apart: (K + 8) additions of terms s (q + z) |x| at most, and
    # the staged x, off by 2^-40 of its row's largest, which 2^-23 of one such term in 2^17 covers
    acc = (K + 8) * 2.0**-23 * (np.abs(f64(x)) @ w4_terms(w).T) + 2.0**-23 * np.abs(ref)
    within(y, ref, acc + 2.0**-8 * (np.abs(ref) + acc), f"w4_linear {rows, K, N, group, zeros, bias}")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,kg,N", [(1, 1, 1), (1, 8, 16), (2, 3, 17), (7, 5, 250), (8, 16, 128), (9, 4, 33),
                                       (16, 7, 48), (17, 2, 64), (31, 9, 136), (33, 8, 15), (70, 3, 40)])
def test_w4_linear(rows, kg, N, group):
    check_linear(rows, kg * group, N, group, zeros=rows % 2 == 0, bias=N % 2 == 0)
    check_linear(rows, kg * group, N, group, zeros=rows % 2 == 1, bias=N % 2 == 1)


@pytest.mark.parametrize("rows,K,N,group", [(1, 4096, 6144, 128), (5, 14336, 512, 64), (40, 1280, 2000, 32)])
def test_w4_linear_larger(rows, K, N, group):
    check_linear(rows, K, N, group, True, True, seed=3)


@pytest.mark.parametrize("rows,K,N,group", [(3, 40960, 40, 32), (8, 4224, 333, 128), (11, 14336, 70, 64),
                                            (24, 5120, 200, 32), (33, 8192, 96, 128), (64, 2176, 33, 64)])
def test_w4_linear_long_rows_of_a_narrow_weight(rows, K, N, group):
    """K split over several CTAs."""
    check_linear(rows, K, N, group, True, False, seed=5)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("rows", [1, 8, 20, 30])
def test_zeros_of_a_weight_stay_zeros(rows, zero_points, group):
    """Rows, and groups of a row, that are zero add exactly nothing."""
    K, N = 5 * group, 70
    w = randn((N, K), 11, K**-0.5)
    w[::3] = 0.0
    w[1, group:] = 0.0
    codes, scales, zeros = dg.w4_quantize(w.to(DEV), group, zero_points)
    x = randn((rows, K), 12) * 100.0
    y = dg.w4_linear(x.to(DEV), codes, scales, zeros)
    assert (y[:, ::3] == 0).all() and (y[:, 1] != 0).all()
    first = slice(0, group)
    alone = dg.w4_linear(x[:, first].contiguous().to(DEV), codes[:, : group // 2].contiguous(),
                         scales[:, :1].contiguous(), None if zeros is None else zeros[:, :1].contiguous())
    ref = few.w4_linear(f64(x), few.w4_values(codes.cpu().numpy(), f64(scales),
                                              None if zeros is None else zeros.cpu().numpy()))
    for got in (y, alone):
        within(got[:, 1], ref[:, 1], 2.0**-8 * np.abs(ref[:, 1]) + 2 * group * 2.0**-23 *
               (15 * f64(scales)[1, 0] * np.abs(f64(x))[:, first].sum(1)), "one group")


def test_wrappers_name_what_is_no_weight():
    x = randn((2, 64), 3).to(DEV)
    w, _ = w4_weight((), 24, 64, 32, False, 4)
    idx, gates = torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
    for call, name in ((lambda: dg.w4_linear(x, None, None), "codes"), (lambda: dg.w4_linear(x, w[0], None), "scales"),
                       (lambda: dg.moe_route(x, [1], 1), "w_router"), (lambda: dg.moe_route(x[0], x, 1), "x"),
                       (lambda: dg.moe_swiglu(x, idx, gates, None, x), "w13"),
                       (lambda: dg.moe_swiglu(x, idx, gates, torch.zeros((1, 16, 64), dtype=BF16, device=DEV), 1), "w2"),
                       (lambda: dg.moe_swiglu_w4(x, idx, gates, (None,) * 3, w), "codes")):
        with pytest.raises((TypeError, ValueError), match=name):
            call()


def test_w4_linear_keeps_nonfinite_values_in_their_row_and_column():
    x = randn((11, 256), 1)
    w, _ = w4_weight((), 40, 256, 64, True, 2)
    clean = dg.w4_linear(x.to(DEV), *w)
    x[3, 7], x[9, 200] = float("nan"), float("inf")
    scales = w[1].clone()
    scales[5, 2] = float("nan")
    y = dg.w4_linear(x.to(DEV), w[0], scales, w[2])
    assert torch.isnan(y[3]).all() and torch.isnan(y[:, 5]).all() and not torch.isfinite(y[9]).any()
    rows = [r for r in range(11) if r not in (3, 9)]
    cols = [c for c in range(40) if c != 5]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])


def test_w4_linear_shapes_and_empty():
    w, _ = w4_weight((), 24, 64, 32, False, 4)
    x = randn((2, 3, 64), 4).to(DEV)
    y = dg.w4_linear(x, *w)
    assert y.shape == (2, 3, 24) and torch.equal(y.view(6, 24), dg.w4_linear(x.view(6, 64), *w))
    assert dg.w4_linear(x[:0], *w).shape == (0, 3, 24)
    out = torch.empty_like(y)
    assert dg.w4_linear(x, *w, out=out) is out and torch.equal(out, y)
    with pytest.raises(ValueError, match="contiguous"):
        dg.w4_linear(x.transpose(0, 1), *w)
    with pytest.raises(ValueError):
        dg.w4_linear(x, w[0], w[1][:, :1].contiguous().expand(24, 3).contiguous())
    with pytest.raises(dg._lib.DGError, match="group"):
        dg.w4_linear(x, w[0], w[1][:, :1].repeat(1, 4))


def test_w4_rows_are_the_same_alone_and_in_a_batch():
    # one row's result does not hang on which rows ride along within a batch of 8
    w, _ = w4_weight((), 80, 512, 128, True, 6)
    x = randn((8, 512), 6).to(DEV)
    y = dg.w4_linear(x, *w)
    for r in (0, 5):
        assert torch.equal(dg.w4_linear(x[r:r + 1].contiguous(), *w)[0], y[r])


# ------------------------------------------------------------------ router

def check_route(x, w, k, score="softmax", renorm=True, scale=1.0):
    idx, gates = dg.moe_route(x.to(DEV), w.to(DEV), k, score=score, renormalize=renorm, scale=scale)
    logits = few.moe_logits(f64(x), f64(w))
    ri, rg = few.moe_choose(logits, k, score, renorm, scale)
    assert idx.dtype == torch.int32 and np.array_equal(idx.cpu().numpy(), ri)
    # each exp is off by 4 * 2^-24 and its argument's rounding, sums of E terms by E * 2^-24, quotient and
    # scale by 2 * 2^-24; a gate below the smallest normal number by that number
    args = np.abs(logits - logits.max(1, keepdims=True)).max() + np.abs(logits).max()
    rel = 2.0**-24 * (logits.shape[1] + 16 + 2 * args)
    g = f64(gates)
    assert np.all(np.abs(g - rg) <= rel * np.abs(rg) + 2.0**-126)


@pytest.mark.parametrize("T,d,E,k", [(1, 8, 1, 1), (1, 4096, 64, 8), (3, 264, 7, 7), (5, 128, 33, 5), (9, 1000, 256, 4),
                                     (130, 64, 128, 6), (2, 512, 1000, 32)])
@pytest.mark.parametrize("score,renorm,scale", [("softmax", True, 1.0), ("softmax", False, 2.5),
                                                ("sigmoid", True, 1.0), ("sigmoid", False, 0.5)])
def test_route(T, d, E, k, score, renorm, scale):
    check_route(randn((T, d), T + d), randn((E, d), E + d, d**-0.5), k, score, renorm, scale)


def test_route_ties_go_to_the_lower_expert():
    w = randn((12, 64), 1)
    w = torch.cat([w, w, w.flip(0)])        # every logit three times
    check_route(randn((6, 64), 2), w, 20)
    check_route(torch.zeros((2, 64), dtype=BF16), w, 7, renorm=False)   # all equal, +0 and -0 alike
    signs = torch.ones((9, 64), dtype=BF16)
    signs[::2] = -1
    check_route(torch.zeros((1, 64), dtype=BF16), signs, 9)


def test_route_cancelling_sums_are_ranked_exactly():
    # logits whose large parts cancel: a sum in plain binary32 would lose the small differences that rank them
    E, d = 16, 64
    w = torch.zeros((E, d))
    w[:, 0], w[:, 1] = 2.0**30, -(2.0**30)
    w[:, 2] = torch.arange(E) * 2.0**-10
    x = torch.ones((1, d))
    check_route(x.to(BF16), w.to(BF16), 5)
    perm = torch.randperm(d, generator=torch.Generator().manual_seed(0))
    check_route(x.to(BF16), w[:, perm].contiguous().to(BF16), 5)


def test_route_nan_and_inf():
    x, w = randn((4, 64), 3), randn((10, 64), 4)
    w[2, 5] = float("nan")                     # expert 2: NaN for every token
    x[1, 9] = float("nan")                     # token 1: all NaN
    for k in (3, 10):
        idx, gates = dg.moe_route(x.to(DEV), w.to(DEV), k)
        i = idx.cpu()
        assert all(len(set(r.tolist())) == k and set(r.tolist()) <= set(range(10)) for r in i)
        assert torch.isnan(gates).all()
        assert i[1].tolist() == list(range(k))
        if k == 10:
            assert (i[[0, 2, 3], -1] == 2).all()
        else:
            assert (i[[0, 2, 3]] != 2).all()


def test_route_empty_and_refusals():
    x, w = randn((2, 64), 3).to(DEV), randn((10, 64), 4).to(DEV)
    idx, gates = dg.moe_route(x[:0], w, 2)
    assert idx.shape == (0, 2) and gates.shape == (0, 2)
    for bad in (0, 11):
        with pytest.raises(dg._lib.DGError, match="k must be"):
            dg.moe_route(x, w, bad)
    with pytest.raises(ValueError, match="workspace"):
        dg.moe_route(x, w, 2, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ experts

def routing(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    gates = torch.rand((T, k), generator=g) + 0.1
    return idx, gates / gates.sum(1, keepdim=True)


def check_moe(T, d, F, E, idx, gates, seed=0, group=0, zeros=False):
    x = randn((T, d), seed + T)
    if group:
        w13, v13 = w4_weight((E,), 2 * F, d, group, zeros, seed + 1)
        w2, v2 = w4_weight((E,), d, F, group, zeros, seed + 2)
        y = dg.moe_swiglu_w4(x.to(DEV), idx.to(DEV), gates.to(DEV), w13, w2)
    else:
        b13, b2 = randn((E, 2 * F, d), seed + 1, d**-0.5), randn((E, d, F), seed + 2, F**-0.5)
        v13, v2 = f64(b13), f64(b2)
        y = dg.moe_swiglu(x.to(DEV), idx.to(DEV), gates.to(DEV), b13.to(DEV), b2.to(DEV))
    i, gt = idx.numpy(), f64(gates)
    ref = few.moe_swiglu(f64(x), i, gt, v13, v2)
    terms = (w4_terms(w13), w4_terms(w2)) if group else ()
    within(y, ref, few.moe_swiglu_bound(f64(x), i, gt, v13, v2, *terms), f"moe {T, d, F, E, group, zeros}")
    # and in the norm: h and y each rounded to bf16, 2^-8 apiece at most
    assert np.linalg.norm(f64(y) - ref) <= 2 * 2.0**-8 * max(np.linalg.norm(ref), 1e-30)
    return y


SHAPES = [(1, 8, 8, 1, 1), (1, 64, 32, 4, 2), (1, 264, 200, 6, 3), (2, 520, 136, 9, 2), (5, 128, 72, 3, 3),
          (8, 72, 512, 8, 1), (20, 256, 104, 4, 2), (33, 136, 264, 5, 4), (64, 96, 48, 2, 2), (100, 64, 40, 3, 1),
          (40, 2056, 24, 16, 8)]


@pytest.mark.parametrize("T,d,F,E,k", SHAPES)
def test_moe_bf16(T, d, F, E, k):
    check_moe(T, d, F, E, *routing(T, E, k, T + E), seed=T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,dg_,Fg,E,k", [(1, 1, 1, 1, 1), (1, 3, 2, 4, 2), (3, 2, 5, 6, 6), (9, 4, 1, 5, 2),
                                          (20, 1, 3, 4, 3), (50, 2, 2, 3, 2)])
def test_moe_w4(T, dg_, Fg, E, k, group):
    check_moe(T, dg_ * group, Fg * group, E, *routing(T, E, k, T + E), seed=T, group=group, zeros=T % 2 == 1)


def test_moe_one_expert_takes_every_token():
    # all pairs land on one expert: several column blocks of one entry
    for T, E in ((90, 64), (9, 300), (200, 1)):
        idx = torch.full((T, 1), E - 1, dtype=torch.int32)
        check_moe(T, 64, 48, E, idx, torch.ones((T, 1)), seed=T)


@pytest.mark.parametrize("group", [0, 64])
def test_moe_padding_repeats_and_foreign_experts(group):
    T, d, F, E, k = 23, 128, 64, 5, 4
    idx, gates = routing(T, E, k, 7)
    idx[3] = -1                                   # a token without experts
    idx[4] = torch.tensor([2, 2, 2, 2])           # one expert four times
    idx[5] = torch.tensor([0, E, -7, 2**31 - 1])  # experts of another rank
    idx[20:] = -1                                 # a padded tail
    y = check_moe(T, d, F, E, idx, gates, seed=9, group=group, zeros=True)
    assert not y[3].any() and not y[20:].any()
    y = check_moe(T, d, F, E, torch.full_like(idx, -1), gates, seed=9, group=group)
    assert not y.any()


def test_moe_nonfinite_values_stay_with_their_token_and_expert():
    T, d, F, E, k = 12, 64, 40, 4, 2
    idx, gates = routing(T, E, k, 8)
    idx[0], idx[1] = torch.tensor([0, 1]), torch.tensor([2, 3])
    x, w13, w2 = randn((T, d), 1), randn((E, 2 * F, d), 2, 0.2), randn((E, d, F), 3, 0.2)
    args = [t.to(DEV) for t in (x, idx, gates, w13, w2)]
    clean = dg.moe_swiglu(*args)
    args[0][5, 3] = float("nan")
    args[3][3, 7, 0] = float("inf")
    y = dg.moe_swiglu(*args)
    hit = (idx == 3).any(1)
    hit[5] = True
    assert torch.isnan(y[5]).all() and torch.equal(y[~hit.to(DEV)], clean[~hit.to(DEV)]) and bool((~hit).any())
    # an expert that no token picked may hold anything
    args[0][5, 3] = 0.0
    args[1] = torch.where(args[1] == 3, torch.full_like(args[1], -1), args[1])
    assert torch.isfinite(dg.moe_swiglu(*args).float()).all()


def test_moe_empty_and_limits():
    x, w13, w2 = randn((4, 64), 1).to(DEV), randn((2, 32, 64), 2).to(DEV), randn((2, 64, 16), 3).to(DEV)
    idx, gates = torch.zeros((4, 1), dtype=torch.int32, device=DEV), torch.ones((4, 1), device=DEV)
    assert dg.moe_swiglu(x[:0], idx[:0], gates[:0], w13, w2).shape == (0, 64)
    big = torch.zeros((8193, 64), dtype=BF16, device=DEV)
    with pytest.raises(dg._lib.DGError, match="split the batch"):
        dg.moe_swiglu(big, torch.zeros((8193, 1), dtype=torch.int32, device=DEV), torch.ones((8193, 1), device=DEV),
                      w13, w2)
    with pytest.raises(TypeError, match="idx"):
        dg.moe_swiglu(x, idx.long(), gates, w13, w2)
    with pytest.raises(ValueError, match="w2"):
        dg.moe_swiglu(x, idx, gates, w13, w2.transpose(1, 2).contiguous())
    with pytest.raises(ValueError, match="same group"):
        a, b = dg.w4_quantize(randn((2, 128, 64), 4).to(DEV), 32), dg.w4_quantize(randn((2, 64, 64), 4).to(DEV), 64)
        dg.moe_swiglu_w4(x, idx, gates, a, b)
    # the largest call: 8192 pairs
    T = 4096
    g = torch.Generator().manual_seed(2)
    idx = torch.randint(-1, 3, (T, 2), generator=g, dtype=torch.int32)
    gates = torch.rand((T, 2), generator=g)
    x = randn((T, 64), 5)
    y = dg.moe_swiglu(x.to(DEV), idx.to(DEV), gates.to(DEV), w13, w2)
    rows = np.r_[0:20, T - 20:T]
    sub = (f64(x)[rows], idx.numpy()[rows], f64(gates)[rows], f64(w13), f64(w2))
    within(y[rows], few.moe_swiglu(*sub), few.moe_swiglu_bound(*sub), "8192 pairs")


# ------------------------------------------------------------------ together, and as calls are made

def test_a_routed_decode_step_together():
    """QKV-style 4-bit projection, its output through the router and the experts, bf16 and 4-bit."""
    T, d, F, E, k, group = 6, 256, 128, 8, 3, 64
    x = randn((T, 128), 1).to(DEV)
    wp, vp = w4_weight((), d, 128, group, False, 2)
    h = dg.w4_linear(x, *wp)
    wr = randn((E, d), 3, d**-0.5).to(DEV)
    b13, b2 = randn((E, 2 * F, d), 4, d**-0.5).to(DEV), randn((E, d, F), 5, F**-0.5).to(DEV)
    q13, q2 = dg.w4_quantize(b13, group), dg.w4_quantize(b2, group)
    idx, gates = dg.moe_route(h, wr, k, scale=1.5)
    ri, rg = few.moe_choose(few.moe_logits(f64(h), f64(wr)), k, scale=1.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    for w13, w2, call in ((b13, b2, dg.moe_swiglu), (q13, q2, dg.moe_swiglu_w4)):
        y = dg.moe_layer(h, wr, w13, w2, k, scale=1.5)
        assert torch.equal(y, call(h, idx, gates, w13, w2))
        v13, v2 = (f64(w) if torch.is_tensor(w) else few.w4_values(w[0].cpu().numpy(), f64(w[1]), None)
                   for w in (w13, w2))
        args = (f64(h), ri, f64(gates), v13, v2)
        terms = () if torch.is_tensor(w13) else (w4_terms(w13), w4_terms(w2))
        within(y, few.moe_swiglu(*args), few.moe_swiglu_bound(*args, *terms), "moe_layer")
    # the dequantised weights through the bf16 layer: the same experts up to the rounding of the values
    y4 = dg.moe_swiglu_w4(h, idx, gates, q13, q2)
    yd = dg.moe_swiglu(h, idx, gates, dg.w4_dequantize(*q13), dg.w4_dequantize(*q2))
    assert (y4.float() - yd.float()).norm() <= 6 * 2.0**-8 * y4.float().norm()


def decode_calls():
    T, d, F, E, k, group = 5, 256, 128, 8, 3, 64
    x, wr = randn((T, d), 1).to(DEV), randn((E, d), 3, d**-0.5).to(DEV)
    b13, b2 = randn((E, 2 * F, d), 4, d**-0.5).to(DEV), randn((E, d, F), 5, F**-0.5).to(DEV)
    q13, q2 = dg.w4_quantize(b13, group, True), dg.w4_quantize(b2, group, True)
    flat = dg.w4_quantize(wr, group)
    return x, {
        "w4_quantize": lambda x: dg.w4_quantize(x, group, True),
        "w4_dequantize": lambda x: dg.w4_dequantize(*flat),
        "w4_linear": lambda x: dg.w4_linear(x, *flat),
        "moe_route": lambda x: dg.moe_route(x, wr, k),
        "moe_layer": lambda x: dg.moe_layer(x, wr, b13, b2, k),
        "moe_layer_w4": lambda x: dg.moe_layer(x, wr, q13, q2, k),
    }


def flat(out):
    return [out] if torch.is_tensor(out) else list(out)


def test_every_call_repeats_bit_for_bit_and_on_another_stream():
    x, calls = decode_calls()
    s = torch.cuda.Stream()
    for name, f in calls.items():
        first = flat(f(x))
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, flat(f(x)))), name
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = flat(f(x))
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(first, other)), name


def test_every_call_is_captured_and_replayed_on_new_inputs():
    x, calls = decode_calls()
    for name, f in calls.items():
        buf = x.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f(buf)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = flat(f(buf))
        for seed in (11, 12):
            buf.copy_(randn(x.shape, seed).to(DEV))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, flat(f(buf.clone())))), name


def test_two_captured_layers_replay_at_the_same_time():
    x, calls = decode_calls()
    f = calls["moe_layer"]
    xs = [randn(x.shape, s).to(DEV) for s in (21, 22)]
    graphs, outs = [], []
    for v in xs:
        f(v)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f(v))
        graphs.append(g)
    want = [f(v) for v in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_skip_their_work_while_the_workspace_holds_an_error():
    x, _ = decode_calls()
    w, _ = w4_weight((), 24, 256, 64, False, 4)
    b13, b2 = randn((4, 64, 256), 4).to(DEV), randn((4, 256, 32), 5).to(DEV)
    idx, gates = (t.to(DEV) for t in routing(5, 4, 2, 1))
    ws = dg.alloc_workspace(1 << 20, DEV)
    calls = [lambda out: dg.w4_linear(x, *w, out=out, ws=ws),
             lambda out: dg.moe_swiglu(x, idx, gates, b13, b2, workspace=ws, out=out)]
    for f, n in zip(calls, (24, 256)):
        out = torch.full((5, n), 7.0, dtype=BF16, device=DEV)
        dg.debug_wait_timeout(5_000, workspace=ws)
        f(out)
        torch.cuda.synchronize()
        assert torch.all(out == 7.0)
        assert dg.device_status(workspace=ws)[0] == 4
        f(out)
        assert not torch.all(out == 7.0) and dg.device_status(workspace=ws)[0] == 0

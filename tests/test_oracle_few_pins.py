"""Pins of the few-token oracle (4-bit weights, routed experts) against
independent formulations."""
import numpy as np
import pytest
import torch

from oracle import few


def test_bf16_rounding_matches_torch():
    g = torch.Generator().manual_seed(0)
    v = torch.cat([torch.randn(20000, generator=g) * 10.0 ** torch.randint(-30, 30, (20000,), generator=g),
                   torch.tensor([0.0, -0.0, float("inf"), float("-inf"), 1.00390625, 1.01171875])])
    got = few.bf16_rne(v.numpy())
    assert np.array_equal(got, v.to(torch.bfloat16).double().numpy())
    assert np.isnan(few.bf16_rne(np.float32(np.nan)))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero_points", [False, True])
def test_quantizer_is_within_half_a_step(group, zero_points):
    g = torch.Generator().manual_seed(group)
    w = torch.randn(7, 256, generator=g).to(torch.bfloat16).double().numpy()
    q, s, z = few.w4_quantize(w, group, zero_points)
    assert q.max() <= 15
    v = few.w4_values(few.w4_pack(q), s, z if zero_points else None)
    step = np.repeat(s, group, axis=1)
    # half a step from rounding; the ends of the range lie up to half a step (zero points) or a
    # bf16 rounding of the scale, 7 * 2^-8 of a step, further out
    assert np.all(np.abs(v - w) <= step * (1.0 + 15 * 2.0**-8 if zero_points else 0.5 + 7 * 2.0**-8))
    assert np.array_equal(few.w4_unpack(few.w4_pack(q)), q)


def test_quantizer_hand_example():
    w = np.zeros((1, 32))
    w[0, :4] = [7.0, -7.0, 2.5, 3.5]      # scale 1: ties go to the even code
    q, s, z = few.w4_quantize(w, 32, False)
    assert s[0, 0] == 1.0 and list(q[0, :5]) == [15, 1, 10, 12, 8]
    w[0, :4] = [10.0, -5.0, 0.0, 1.0]     # range 15: scale 1, zero point 5
    q, s, z = few.w4_quantize(w, 32, True)
    assert s[0, 0] == 1.0 and z[0, 0] == 5 and list(q[0, :5]) == [15, 0, 5, 6, 5]
    q, s, z = few.w4_quantize(np.zeros((1, 32)), 32, True)
    assert s[0, 0] == 1.0 and z[0, 0] == 0 and not q.any()
    w[0, 3] = np.nan
    q, s, z = few.w4_quantize(w, 32, True)
    assert np.isnan(s[0, 0]) and z[0, 0] == 8


def test_choice_against_torch():
    g = torch.Generator().manual_seed(3)
    l = torch.randn(40, 24, generator=g)
    l[::2] = torch.round(l[::2] * 2) / 2   # many ties
    for score in ("softmax", "sigmoid"):
        p = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :5]
        for renorm in (True, False):
            want = torch.gather(p, 1, order)
            want = (want / want.sum(1, keepdim=True) if renorm else want) * 1.5
            idx, gates = few.moe_choose(l.double().numpy(), 5, score, renorm, 1.5)
            assert np.array_equal(idx, order.numpy())
            np.testing.assert_allclose(gates, want.numpy(), rtol=1e-14)
    l[0, 3] = float("nan")
    idx, gates = few.moe_choose(l.double().numpy()[:1], 24)
    assert idx[0, -1] == 3 and np.isnan(gates).all() and sorted(idx[0]) == list(range(24))


def test_experts_against_torch():
    g = torch.Generator().manual_seed(4)
    T, d, F, E, k = 6, 16, 24, 5, 3
    x, w13, w2 = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((T, d), (E, 2 * F, d), (E, d, F)))
    idx = torch.randint(-1, E + 1, (T, k), generator=g)   # some outside [0, E), some twice
    idx[0] = -1
    gates = torch.rand(T, k, generator=g, dtype=torch.float64)
    got = few.moe_swiglu(x.numpy(), idx.numpy(), gates.numpy(), w13.numpy(), w2.numpy())
    share = torch.zeros(T, E + 2, dtype=torch.float64)
    share.scatter_add_(1, torch.where((idx < 0) | (idx >= E), E + 1, idx), gates)
    a, b = torch.einsum("td,efd->tef", x, w13).chunk(2, dim=2)
    want = torch.einsum("tef,edf,te->td", torch.nn.functional.silu(a) * b, w2, share[:, :E])
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-10, atol=1e-10)
    assert not got[0].any()
    bound = few.moe_swiglu_bound(x.numpy(), idx.numpy(), gates.numpy(), w13.numpy(), w2.numpy())
    routed = ((idx >= 0) & (idx < E)).any(1).numpy()
    assert not routed[0] and routed.any()
    assert np.all(bound[routed] > 0) and np.all(bound[~routed] == 0)

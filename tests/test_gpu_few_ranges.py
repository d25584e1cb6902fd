"""Few-token operators on values far apart: activations that span more than the staged form holds,
weights near the smallest numbers, logits whose sigmoids are below them."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import few
from test_gpu_few import BF16, DEV, check_route, f64, randn, w4_terms, w4_weight, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 5, 9, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("small", [2.0**-3, 2.0**-9, 2.0**-14, 2.0**-22])
def test_a_large_activation_on_a_zero_weight(rows, group, small):
    """Activations 2^23 to 2^42 times smaller than their row's largest, which meets codes and zero points of 0."""
    K, N = 2 * group if group > 32 else 160, 40
    x = randn((rows, K), rows) * small
    x[:, 0] = 2.0**20
    (codes, scales, zeros), _ = w4_weight((), N, K, group, True, 4)
    codes[:, 0] &= 0xF0      # column 0, the low nibble: code 0
    zeros[:, 0] = 0          # of its group
    y = dg.w4_linear(x.to(DEV), codes, scales, zeros)
    xs, z, s = f64(x), zeros.cpu().numpy(), f64(scales)
    ref = few.w4_linear(xs, few.w4_values(codes.cpu().numpy(), s, z))
    # (K + 8) additions of terms s (q + z) |x| at most; activations held to 2^-35 of the largest in s q x
    acc = (K + 8) * 2.0**-23 * (np.abs(xs) @ w4_terms((codes, scales, zeros)).T)
    held = 2.0**-35 * np.abs(xs).max(1, keepdims=True) * few.w4_values(codes.cpu().numpy(), s, 0 * z).sum(1)
    acc = acc + held + 2.0**-23 * np.abs(ref)
    within(y, ref, acc + 2.0**-8 * (np.abs(ref) + acc), f"{rows, group, small}")


@pytest.mark.parametrize("rows", [1, 8, 9, 33])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("weight,activation", [(-131, 0), (-126, 0), (-100, -24), (-40, -90), (-133, 12), (-10, -110),
                                               (120, -122), (100, -130), (1, 120)])
def test_w4_linear_of_tiny_and_huge_values(rows, group, weight, activation):
    """Scales around 2^weight on activations around 2^activation, products down to bf16's subnormal numbers."""
    K, N = 2 * group, 40
    x = (randn((rows, K), rows).float() * 2.0**activation).to(BF16)
    (codes, scales, zeros), _ = w4_weight((), N, K, group, True, 4)
    scales = torch.ldexp(scales.double() * (4 * K**0.5), torch.tensor(weight, device=DEV)).to(BF16)    # 0.5 to 1.5 before
    y = dg.w4_linear(x.to(DEV), codes, scales, zeros)
    w = (codes, scales, zeros)
    ref = few.w4_linear(f64(x), few.w4_values(codes.cpu().numpy(), f64(scales), zeros.cpu().numpy()))
    # as elsewhere; then what 32-bit numbers below 2^-126 lose: half of 2^-149 for each of at most 8 group sums
    # (K / group and the slices' joins) and for the factor's product, in units of 2^-14 of the row's largest
    # and of 1; and half a step of bf16's, 2^-133
    xs = f64(x)
    acc = (K + 8) * 2.0**-23 * (np.abs(xs) @ w4_terms(w).T) + 2.0**-23 * np.abs(ref)
    acc = acc + 2.0**-150 * 2.0**14 * (8 * np.maximum(np.abs(xs).max(1, keepdims=True), 1.0) + 1)
    bound = acc + 2.0**-8 * (np.abs(ref) + acc) + 2.0**-134
    # the largest: 64 to 256 terms of 2^1 * 2^120 * (q - z) can add up to more than binary32 holds
    holds = np.abs(ref) + bound < 2.0**127
    assert holds.mean() > 0.25
    within(torch.where(torch.from_numpy(holds).to(DEV), y, 0.0), np.where(holds, ref, 0.0), bound,
           f"{rows, group, weight, activation}")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("near,far", [(-60.0, -60.0), (-95.0, -95.0), (-150.0, -150.0), (-1000.0, -1000.0),
                                      (-20.0, -110.0), (30.0, -100.0), (200.0, 100.0)])
def test_route_sigmoids_of_large_logits(near, far, renorm):
    """Logits around `near` for every other expert and around `far` for the rest."""
    d, E = 64, 24
    w = randn((E, d), 5, 0.25).float()
    w[::2] += near / d
    w[1::2] += far / d
    x = torch.ones((3, d)) + 0.125 * torch.arange(3)[:, None]
    check_route(x.to(BF16), w.to(BF16), 16, "sigmoid", renorm, 2.5)
    _, gates = dg.moe_route(x.to(BF16).to(DEV), w.to(BF16).to(DEV), 16, score="sigmoid", renormalize=renorm)
    if renorm:   # 16 gates that add up to 1, each off by a few units, and so the sum
        assert torch.isfinite(gates).all() and (gates.sum(1) - 1).abs().max() <= 16 * 2.0**-22

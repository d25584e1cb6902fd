"""Expert products whose CTAs take several units, of changing width: more units than CTAs, experts
of 1 to 35 tokens side by side, row blocks that do not fill the last CTA, K split 1, 2 and 4 ways.

A unit's shared memory is laid out by its width, so a warp that runs ahead into the next unit
may not write there before the others have left the last one."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import few
from test_gpu_few import DEV, f64, randn, w4_terms, w4_weight, within

pytestmark = pytest.mark.gpu

WIDE = (1, 3, 5, 8, 9, 14, 17, 20, 25, 30, 32, 35)
TWO = (1, 2, 5, 8, 9, 12, 16)


def uneven_routing(T, k, E, sizes, seed):
    """idx [T, k] that gives expert e a number of tokens drawn from `sizes`; what is left over is -1."""
    rng = np.random.default_rng(seed)
    idx, free = np.full((T, k), -1, dtype=np.int32), np.full(T, k)
    for e in range(E):
        n = min(int(rng.choice(sizes)), int((free > 0).sum()))
        # the tokens with the most choices left, ties at random
        for t in sorted(range(T), key=lambda t: (-free[t], rng.random()))[:n]:
            idx[t, k - free[t]] = e
            free[t] -= 1
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(seed)) + 0.1
    return torch.from_numpy(idx), gates / k


def check_units(T, k, E, d, F, sizes, group=0, repeats=50):
    idx, gates = uneven_routing(T, k, E, sizes, T + E)
    x = randn((T, d), 1)
    if group:
        w13, v13 = w4_weight((E,), 2 * F, d, group, True, 2)
        w2, v2 = w4_weight((E,), d, F, group, True, 3)
        terms = (w4_terms(w13), w4_terms(w2))
        call = dg.moe_swiglu_w4
    else:
        w13, w2 = randn((E, 2 * F, d), 2, d**-0.5).to(DEV), randn((E, d, F), 3, F**-0.5).to(DEV)
        v13, v2, terms, call = f64(w13), f64(w2), (), dg.moe_swiglu
    args = (x.to(DEV), idx.to(DEV), gates.to(DEV), w13, w2)
    y = call(*args)
    ref, bound = few.moe_swiglu_by_expert(f64(x), idx.numpy(), f64(gates), v13, v2, *terms)
    within(y, ref, bound, f"{T, k, E, d, F, group}")
    # h and y are each rounded to bf16, 2^-8 apiece at most
    assert np.linalg.norm(f64(y) - ref) <= 2 * 2.0**-8 * np.linalg.norm(ref)
    for _ in range(repeats):
        assert torch.equal(call(*args), y)


@pytest.mark.parametrize("E,k,d,F,sizes,group", [
    (56, 16, 288, 1312, WIDE, 32),       # up: whole K a warp, 2 of 8 row blocks idle in the last CTA of an expert
    (56, 16, 2880, 96, WIDE, 32),        # down: the same
    (100, 28, 512, 1088, WIDE, 32),      # down: K split 2 ways
    (100, 28, 512, 1152, WIDE, 128),
    (64, 8, 1088, 832, TWO, 64),         # up to 16 pairs: up whole, down split 2 ways
])
def test_4_bit_units_of_changing_width(E, k, d, F, sizes, group):
    check_units(64, k, E, d, F, sizes, group)


@pytest.mark.parametrize("E,k,d,F,sizes", [
    (56, 16, 264, 1304, WIDE),           # up: K split 2 ways
    (56, 16, 1304, 264, WIDE),           # down: whole K a warp
    (64, 8, 520, 1048, TWO),             # up whole, down split 4 ways
    (64, 8, 1048, 520, TWO),             # both split 2 ways
])
def test_bf16_units_of_changing_width(E, k, d, F, sizes):
    check_units(64, k, E, d, F, sizes)


@pytest.mark.parametrize("k,E,d,F,group", [(8, 8, 64, 16384, 0), (8, 8, 16384, 64, 0), (32, 32, 128, 4096, 32),
                                           (32, 32, 4096, 128, 128)])
def test_one_token_with_more_units_than_ctas(k, E, d, F, group):
    """Every CTA builds the map, and (4 bits) stages the rows of each unit, itself."""
    check_units(1, k, E, d, F, (1,), group, repeats=20)

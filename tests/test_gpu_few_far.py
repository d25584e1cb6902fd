"""Few-token operators on tensors whose offsets pass 2^31 elements or 2^32 bytes, and on the most rows they take."""
import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import few
from test_gpu_few import BF16, DEV, f64, randn, routing, w4_terms, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def gpu_gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def linear_bound(x, w, ref):
    """As in test_gpu_few.check_linear."""
    acc = (x.shape[1] + 8) * 2.0**-23 * (np.abs(x) @ w4_terms(w).T) + 2.0**-23 * np.abs(ref)
    return acc + 2.0**-8 * (np.abs(ref) + acc)


@pytest.mark.parametrize("rows", [1, 9])
def test_w4_linear_codes_beyond_4_gib(rows):
    N, K, group = 140001, 65536, 128
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gpu_gen(1))
    scales = (torch.rand((N, K // group), device=DEV, generator=gpu_gen(2)) + 0.5).div_(4 * K**0.5).to(BF16)
    x = randn((rows, K), 3)
    y = dg.w4_linear(x.to(DEV), codes, scales)
    for n in (0, 65535, 131071, 139990):    # codes pass 2^31 bytes at row 65536, 2^32 at 131072
        part = slice(n, n + 11)
        w = (codes[part].clone(), scales[part].clone(), None)
        ref = few.w4_linear(f64(x), few.w4_values(w[0].cpu().numpy(), f64(w[1]), None))
        within(y[:, part], ref, linear_bound(f64(x), w, ref), f"rows {n}")


def test_w4_quantize_and_dequantize_beyond_4_gib():
    rows, K, group = 33000, 65536, 64       # 2^31 weights at row 32768
    w = torch.empty((rows, K), dtype=BF16, device=DEV).normal_(generator=gpu_gen(4))
    codes, scales, zeros = dg.w4_quantize(w, group, zero_points=True)
    back = dg.w4_dequantize(codes, scales, zeros)
    for n in (0, 16383, 32767, 32997):
        part = slice(n, n + 3)
        q, s, z = few.w4_quantize(f64(w[part]), group, True)
        assert np.array_equal(codes[part].cpu().numpy(), few.w4_pack(q)) and np.array_equal(f64(scales[part]), s)
        assert np.array_equal(zeros[part].cpu().numpy(), z)
        want = few.bf16_rne(few.w4_values(few.w4_pack(q), s, z).astype(np.float32))
        assert np.array_equal(f64(back[part]), want)


@pytest.mark.parametrize("T", [2, 30])
@pytest.mark.parametrize("group", [0, 32])
def test_experts_beyond_4_gib(T, group):
    E, d, F, k = (260, 2048, 2048, 3) if not group else (1024, 2048, 2080, 3)
    picked = [0, 1, E // 2, E - 130, E - 2, E - 1]
    local, gates = routing(T, len(picked), k, 5)
    idx = torch.tensor(picked, dtype=torch.int32)[local.long()]
    x = randn((T, d), 6)
    if group:
        def weight(n, K, seed):
            codes = torch.randint(0, 256, (E, n, K // 2), dtype=torch.uint8, device=DEV, generator=gpu_gen(seed))
            scales = torch.rand((E, n, K // group), device=DEV, dtype=BF16, generator=gpu_gen(seed + 1))
            return codes, (scales + 0.5).div_(4 * K**0.5), None
        w13, w2 = weight(2 * F, d, 7), weight(d, F, 9)
        y = dg.moe_swiglu_w4(x.to(DEV), idx.to(DEV), gates.to(DEV), w13, w2)
        own = [[(w[0][e], w[1][e], None) for e in picked] for w in (w13, w2)]
        values = [[few.w4_values(c.cpu().numpy(), f64(s), None) for c, s, _ in w] for w in own]
        terms = [[w4_terms(w) for w in ws] for ws in own]
    else:
        w13 = torch.empty((E, 2 * F, d), dtype=BF16, device=DEV).normal_(0, d**-0.5, generator=gpu_gen(7))
        w2 = torch.empty((E, d, F), dtype=BF16, device=DEV).normal_(0, F**-0.5, generator=gpu_gen(8))
        y = dg.moe_swiglu(x.to(DEV), idx.to(DEV), gates.to(DEV), w13, w2)
        values, terms = [[f64(w[e]) for e in picked] for w in (w13, w2)], ()
    ref, bound = few.moe_swiglu_by_expert(f64(x), local.numpy(), f64(gates), *values, *terms)
    within(y, ref, bound, f"{T, group}")


def test_the_most_tokens_of_a_router():
    T, d, E, k = 65535 * 4, 64, 12, 3
    x, w = torch.empty((T, d), dtype=BF16, device=DEV).normal_(generator=gpu_gen(1)), randn((E, d), 2)
    idx, gates = dg.moe_route(x, w.to(DEV), k)
    for t in (0, T // 2 + 1, T - 50):
        rows = slice(t, t + 50)
        i, g = dg.moe_route(x[rows].clone(), w.to(DEV), k)
        ri, rg = few.moe_choose(few.moe_logits(f64(x[rows]), f64(w)), k)
        assert torch.equal(idx[rows], i) and np.array_equal(i.cpu().numpy(), ri)
        # other splits of d round the gates' logits alike; exp and quotient as in test_gpu_few.check_route
        assert np.abs(f64(gates[rows]) - rg).max() <= 2.0**-24 * (E + 16 + 4 * 64) and torch.equal(gates[rows], g)


def test_the_most_rows_of_a_4_bit_linear():
    rows, K, N, group = 65535 * 32, 32, 24, 32
    x = torch.empty((rows, K), dtype=BF16, device=DEV).normal_(generator=gpu_gen(3))
    w = (torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gpu_gen(4)),
         (torch.rand((N, 1), device=DEV, generator=gpu_gen(5)) + 0.5).to(BF16), None)
    y = dg.w4_linear(x, *w)
    values = few.w4_values(w[0].cpu().numpy(), f64(w[1]), None)
    for r in (0, rows // 2 + 5, rows - 70):
        part = f64(x[r:r + 70])
        ref = few.w4_linear(part, values)
        within(y[r:r + 70], ref, linear_bound(part, w, ref), f"rows {r}")

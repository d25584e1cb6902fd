"""The block-scaled linear's backward in scratch of the gradients asked for: the bytes that it says, and no more."""
import itertools

import pytest
import torch

import expert_gemm_layers_gb300 as dg
from expert_gemm_layers_gb300 import _lib
from test_gpu_fp8 import BF16, DEV, randn
from test_gpu_fp8_guards import p, stream
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu
SOME = [n for n in itertools.product((False, True), repeat=3) if any(n)]


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (33, 272, 144), (300, 400, 688), (2060, 144, 272)])
def test_between_guards(rows, K, N):
    lib = _lib.load()
    (xc, xs), (wc, wscale) = dg.fp8_quantize(randn((rows, K), 1).to(DEV)), dg.fp8_quantize(randn((N, K), 2).to(DEV), 128)
    dy = randn((rows, N), 3).to(DEV)
    every = dg.fp8_linear_backward((xc, xs), (wc, wscale), dy, need_db=True)
    for need in SOME:
        g = Guarded()
        out = [g.tensor(s, BF16) if n else None for n, s in zip(need, ((rows, K), (N, K), (N,)))]
        size = lib.dg_fp8_linear_bwd_workspace_bytes_for(rows, K, N, *need)
        ws = g.workspace(size)
        _lib.check(lib.dg_fp8_linear_bwd(rows, K, N, p(xc), p(xs), p(wc), p(wscale), p(dy), *map(p, out), p(ws), size, stream()))
        g.check(f"fp8_linear_bwd {rows, K, N} {need}")
        assert all(t is None or torch.equal(t, every[n]) for t, n in zip(out, ("x", "weight", "bias")))


def test_memory_of_a_call():
    """Beside its gradients a call allocates what these need: with a frozen weight no x in bf16, with a frozen input no
    8-bit dy and no weight."""
    rows, K, N = 4096, 8192, 4096
    x8, w8 = dg.fp8_quantize(randn((rows, K), 1).to(DEV)), dg.fp8_quantize(randn((N, K), 2).to(DEV), 128)
    dy = randn((rows, N), 3).to(DEV)
    for need, outputs, scratch in (((True, False, False), 2 * rows * K, rows * N * 129 // 128 + N * K),
                                   ((False, True, False), 2 * N * K, 2 * rows * K),
                                   ((False, False, True), 2 * N, 4 * N * 1216)):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        dg.fp8_linear_backward(x8, w8, dy, *need)
        torch.cuda.synchronize()
        assert torch.cuda.max_memory_allocated() - before <= outputs + scratch + (4 << 20), need   # torch rounds blocks up

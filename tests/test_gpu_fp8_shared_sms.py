"""Few-row products whose K is split over a cluster, while kernels of other streams wait for their SMs.

With tiles of 64 and 128 rows a CTA sends its sums to its cluster out of its own shared memory.  That memory may go
to the next CTA only when the copies have been read out: results stay those of the calls alone, bit for bit."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from test_gpu_fp8 import DEV, randn

pytestmark = pytest.mark.gpu

# 33 to 512 rows; K split two, four and eight ways
SPLIT = [(40, 640, 272), (33, 2064, 1040), (64, 4096, 6144), (40, 8208, 272), (100, 8192, 528), (128, 14336, 1040),
         (65, 4112, 2064), (300, 12288, 272), (500, 4096, 272)]


@pytest.mark.parametrize("rows,K,N", SPLIT)
def test_split_products_beside_other_streams(rows, K, N):
    ops = [(dg.fp8_quantize(randn((rows, K), s).to(DEV)), dg.fp8_quantize(randn((N, K), s + 9, K**-0.5).to(DEV), 128))
           for s in range(4)]
    x, w = randn((1024, 1040), 20).to(DEV), randn((2064, 1040), 21, 0.03).to(DEV)   # bf16 tiles that fill an SM
    alone = [dg.fp8_linear(*o) for o in ops]
    other = dg.tp_linear(x, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    got = [[] for _ in ops]
    wide = []
    for _ in range(30):
        for o, st, to in zip(ops, streams, got):
            with torch.cuda.stream(st):
                to.append(dg.fp8_linear(*o))
        with torch.cuda.stream(streams[4]):
            wide.append(dg.tp_linear(x, w))
    torch.cuda.synchronize()
    for a, to in zip(alone, got):
        assert all(torch.equal(a, y) for y in to)
    assert all(torch.equal(other, y) for y in wide)
    assert dg.device_status()[0] == 0


@pytest.mark.parametrize("rows,K,N", SPLIT)
def test_split_products_back_to_back(rows, K, N):
    """One stream: the next call's CTAs are let in while the last one's still send."""
    ops = [(dg.fp8_quantize(randn((rows, K), s).to(DEV)), dg.fp8_quantize(randn((N, K), s + 9, K**-0.5).to(DEV), 128))
           for s in range(3)]
    alone = []
    for o in ops:
        alone.append(dg.fp8_linear(*o))
        torch.cuda.synchronize()
    got = [dg.fp8_linear(*ops[i % 3]) for i in range(120)]
    assert all(torch.equal(alone[i % 3], y) for i, y in enumerate(got))

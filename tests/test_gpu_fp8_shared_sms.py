"""Block-scaled products whose CTAs work on one another's shared memory, while kernels of other streams wait for their SMs.

Few rows with K split: with tiles of 64 and 128 rows a CTA sends its sums to its cluster out of its own shared memory,
which may go to the next CTA only when the copies have been read out.  CTA pairs: the second CTA's warps arrive on
barriers of the first, which may go only when they have.  Results stay those of the calls alone, bit for bit."""
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


# tiles of CTA pairs; with 256 n + 1 to 128 rows the last tile's second CTA has none and arrives at once
PAIRS = [(513, 272, 688), (1300, 272, 4112), (600, 2064, 240), (257, 384, 688), (2049, 400, 2064)]


@pytest.mark.parametrize("rows,K,N", PAIRS)
def test_pairs_beside_other_streams(rows, K, N):
    ops = [(dg.fp8_quantize(randn((rows, K), s).to(DEV)), dg.fp8_quantize(randn((N, K), s + 9, K**-0.5).to(DEV), 128),
            randn((rows, N), s + 5).to(DEV)) for s in range(3)]

    def step(x8, w8, dy):
        return dg.fp8_linear(x8, w8), dg.fp8_linear_backward(x8, w8, dy, need_dw=False)["x"]

    x, w = randn((1024, 1040), 20).to(DEV), randn((2064, 1040), 21, 0.03).to(DEV)
    alone = [step(*o) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[] for _ in ops]
    for _ in range(30):
        for o, st, to in zip(ops, streams, got):
            with torch.cuda.stream(st):
                to.append(step(*o))
        with torch.cuda.stream(streams[3]):
            dg.tp_linear(x, w)
    torch.cuda.synchronize()
    for a, to in zip(alone, got):
        assert all(torch.equal(a[0], y) and torch.equal(a[1], dx) for y, dx in to)

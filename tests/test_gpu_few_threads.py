"""Few-token operators called by several threads on one stream, with the module's own workspace."""
import threading

import pytest
import torch

import expert_gemm_layers_gb300 as dg
from test_gpu_few import DEV, randn

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream_get_their_own_results():
    d, F, E, k, group = 256, 128, 24, 4, 64
    wr = randn((E, d), 3, d**-0.5).to(DEV)
    b13, b2 = randn((E, 2 * F, d), 4, d**-0.5).to(DEV), randn((E, d, F), 5, F**-0.5).to(DEV)
    q13, q2 = dg.w4_quantize(b13, group), dg.w4_quantize(b2, group)
    qr = dg.w4_quantize(wr, group)
    xs = [randn((T, d), T).to(DEV) for T in (1, 12, 40, 90)]    # workspaces of other sizes and layouts

    def step(x):
        return [dg.moe_layer(x, wr, b13, b2, k), dg.moe_layer(x, wr, q13, q2, k), dg.w4_linear(x, *qr)]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    got = [None] * len(xs)

    def work(i):
        got[i] = [step(xs[i]) for _ in range(50)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, steps in enumerate(got):
        assert steps is not None and all(torch.equal(a, b) for s in steps for a, b in zip(s, want[i])), xs[i].shape

"""Block-scaled e4m3 operators as a program uses them: chained, on other streams, from threads, captured and replayed."""
import threading

import numpy as np
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from oracle import fp8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16).to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


def weights(d, F):
    q = lambda shape, seed: dg.fp8_quantize(randn(shape, seed, shape[1] ** -0.5), 128)
    return dict(n1=randn((d,), 1), wqkv=q((2 * d, d), 2), wo=q((d, 2 * d), 3), n2=randn((d,), 4), w1=q((F, d), 5),
                w2=q((d, F), 6))


def block(x, stream, w):
    """Two norms with the residual's addition and four products, as one block of a decoder has them (bar attention)."""
    n8, stream = dg.rms_norm(x, w["n1"], stream, fp8=True)
    o = dg.fp8_linear(dg.fp8_linear(n8, w["wqkv"]), w["wo"])
    n8, stream = dg.rms_norm(o, w["n2"], stream, fp8=True)
    return dg.fp8_linear(dg.fp8_linear(n8, w["w1"]), w["w2"]), stream


def plain_block(x, stream, w):
    """The same in binary64 with the operators' own roundings, stage by stage from this run's rounded values."""
    bf = lambda v: fp8.bf16_rne(v.astype(np.float32))
    val = lambda pair: fp8.values(pair[0].cpu().view(torch.uint8).numpy(), pair[1].cpu().view(torch.uint8).numpy(), 128)
    q = lambda v: fp8.values(*fp8.quantize(v))
    h = fp8.add(f64(x), f64(stream))
    o = bf(q(bf(q(fp8.rms_norm(h, f64(w["n1"]), 1e-6)) @ val(w["wqkv"]).T)) @ val(w["wo"]).T)
    h = fp8.add(o, h)
    return bf(q(bf(q(fp8.rms_norm(h, f64(w["n2"]), 1e-6)) @ val(w["w1"]).T)) @ val(w["w2"]).T), h


@pytest.mark.parametrize("rows", [1, 3, 70, 300])
def test_block(rows):
    w = weights(256, 640)
    x, s = randn((rows, 256), 7), randn((rows, 256), 8)
    y, h = block(x, s, w)
    ref, href = plain_block(x, s, w)
    # a value near a border rounds either way: a step of e4m3 (2^-3 of it) in one of 256 terms and more, of which few
    # do; in the 2-norm a hundredth is far more than that, and far less than a wrong scale or row would give
    assert np.linalg.norm(f64(h) - href) <= 1e-2 * np.linalg.norm(href)
    assert np.linalg.norm(f64(y) - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("rows", [1, 24, 260])
def test_captured_blocks_replay(rows):
    """Two graphs captured on one stream and replayed in turn on inputs that change in place."""
    w, st = weights(256, 640), torch.cuda.Stream()
    xs = [randn((rows, 256), 10 + i) for i in range(2)]
    ss = [randn((rows, 256), 20 + i) for i in range(2)]
    graphs, outs = [], []
    with torch.cuda.stream(st):
        block(xs[0], ss[0], w)
        st.synchronize()
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs.append(block(xs[i], ss[i], w))
            graphs.append(g)
    for k in range(3):
        for i in range(2):
            xs[i].copy_(randn((rows, 256), 100 + 2 * k + i))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            y, h = block(xs[i], ss[i], w)
            assert torch.equal(outs[i][0], y) and torch.equal(outs[i][1], h)


def test_captured_training_step():
    x, nw, w = (t.requires_grad_() for t in (randn((90, 272), 1), randn((272,), 2), randn((304, 272), 3, 0.06)))
    r, dy, dh = randn((90, 272), 4), randn((90, 304), 5), randn((90, 272), 6)

    def step():
        out = dg.fp8_norm_linear_layer(x, nw, w, None, r)
        return (*out, *torch.autograd.grad(out, (x, nw, w), (dy, dh)))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = step()
    with torch.no_grad():
        x.copy_(randn((90, 272), 9))
        w.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_streams_and_threads():
    """Calls on several streams and from several threads at once give what they give alone."""
    w = weights(256, 640)
    rows = (1, 20, 140, 300)
    ins = [(randn((n, 256), 30 + n), randn((n, 256), 40 + n)) for n in rows]
    alone = [block(*i, w) for i in ins]
    torch.cuda.synchronize()
    bad = []

    def work(i, own):
        with torch.cuda.stream(torch.cuda.Stream() if own else torch.cuda.default_stream()):
            for _ in range(20):
                y, h = block(*ins[i], w)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(y, alone[i][0]) and torch.equal(h, alone[i][1])):
                    bad.append((i, own))

    for own in (True, False):
        threads = [threading.Thread(target=work, args=(i, own)) for i in range(len(rows))]
        [t.start() for t in threads]
        [t.join() for t in threads]
    assert not bad


def test_rows_behind_the_last_are_left():
    """Outputs are views into larger buffers: nothing past their end is written."""
    for rows, K, N in ((1, 272, 304), (5, 128, 240), (130, 144, 464), (300, 512, 240)):
        buf = torch.full((rows + 300, N), 7.0, dtype=BF16, device=DEV)
        x, w8 = randn((rows, K), 1), dg.fp8_quantize(randn((N, K), 2), 128)
        dg.fp8_linear(x, w8, out=buf[:rows])
        assert (buf[rows:] == 7).all() and not (buf[:rows] == 7).all()
        guard = torch.full((rows + 8, K), 7.0, dtype=BF16, device=DEV)
        dg.fp8_dequantize(*dg.fp8_quantize(x), out=guard[:rows])
        assert (guard[rows:] == 7).all()


def test_same_result_every_time():
    for rows in (1, 30, 300, 2000):
        x, w8 = randn((rows, 2064), 1), dg.fp8_quantize(randn((1040, 2064), 2), 128)
        dy = randn((rows, 1040), 3)
        x8 = dg.fp8_quantize(x)
        y, g = dg.fp8_linear(x8, w8), dg.fp8_linear_backward(x8, w8, dy, need_db=True)
        for _ in range(5):
            assert torch.equal(dg.fp8_linear(x8, w8), y)
            again = dg.fp8_linear_backward(x8, w8, dy, need_db=True)
            assert all(torch.equal(again[n], g[n]) for n in g)

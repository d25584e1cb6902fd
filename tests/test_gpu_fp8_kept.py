"""What the block-scaled layers keep for the backward, and run in it, where only some gradients are asked for."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from test_gpu_fp8 import BF16, DEV, randn

pytestmark = pytest.mark.gpu
ROWS, K, N = 70, 272, 176


def inputs(names):
    made = dict(x=randn((ROWS, K), 1), nw=randn((K,), 2), w=randn((N, K), 3, 0.1), b=randn((N,), 4), r=randn((ROWS, K), 5))
    return {n: t.to(DEV).requires_grad_(n in names) for n, t in made.items()}


def call(layer, t):
    """(outputs, bytes kept beside the inputs themselves)"""
    kept = []
    own = {v.data_ptr() for v in t.values()}
    with torch.autograd.graph.saved_tensors_hooks(lambda v: (kept.append(v), v)[1], lambda v: v):
        out = dg.fp8_linear_layer(t["x"], t["w"], t["b"]) if layer == "linear" else \
            dg.fp8_norm_linear_layer(t["x"], t["nw"], t["w"], t["b"], t["r"])
    out = out if isinstance(out, tuple) else (out,)
    own |= {o.data_ptr() for o in out}   # the residual stream that a layer returns
    return out, sum(v.numel() * v.element_size() for v in kept if v.data_ptr() not in own)


X8, W8 = ROWS * (K + 3), N * K + 2 * 3


@pytest.mark.parametrize("layer,trained,held", [
    ("linear", "x", W8), ("linear", "w", X8), ("linear", "b", 0), ("linear", "wb", X8), ("linear", "xb", W8),
    ("norm", "w", X8), ("norm", "b", 0), ("norm", "wb", X8), ("norm", "x", W8), ("norm", ("nw",), W8), ("norm", "rw", X8 + W8)])
def test_kept_and_gradients(layer, trained, held):
    names = tuple(trained)
    t = inputs(("x", "w", "b") if layer == "linear" else ("x", "nw", "w", "b", "r"))
    dys = [randn((ROWS, N), 6).to(DEV), randn((ROWS, K), 7).to(DEV)]
    out, _ = call(layer, t)
    leaves = [n for n in t if t[n].requires_grad]
    every = dict(zip(leaves, torch.autograd.grad(out, [t[n] for n in leaves], dys[:len(out)])))
    t = inputs(names)
    out, kept = call(layer, t)
    assert kept == held
    some = torch.autograd.grad([o for o in out if o.requires_grad], [t[n] for n in names], dys[:sum(o.requires_grad for o in out)])
    for n, g in zip(names, some):
        assert torch.equal(g, every[n]), n


def launches(run):
    dg.trace_begin()
    try:
        got = run()
    finally:
        seen = dg.trace_end()
    return got, sum(e["launches"] for e in seen)


@pytest.mark.parametrize("layer", ["rms_norm", "norm"])
def test_gradient_of_the_sum_alone(layer):
    """Where nothing came back through the layer's result, h's gradient is passed on and nothing runs."""
    names = ("x", "nw", "r") if layer == "rms_norm" else ("x", "nw", "w", "b", "r")
    t = inputs(names)
    h = (dg.rms_norm_layer(t["x"], t["nw"], t["r"]) if layer == "rms_norm" else call(layer, t)[0])[1]
    dh = randn((ROWS, K), 7).to(DEV)
    got, n = launches(lambda: torch.autograd.grad(h, [t[n] for n in names], dh))
    assert n == 0
    for name, g in zip(names, got):
        assert g.dtype == BF16 and g.shape == t[name].shape
        assert torch.equal(g, dh) if name in "xr" else not g.any()
    # from a broadcast gradient, and into .grad of leaves: theirs alone
    t = inputs(names)
    h = (dg.rms_norm_layer(t["x"], t["nw"], t["r"]) if layer == "rms_norm" else call(layer, t)[0])[1]
    h.sum().backward()
    assert (t["x"].grad == 1).all() and (t["r"].grad == 1).all()
    t["x"].grad.zero_()
    assert (t["r"].grad == 1).all()


def test_bias_gradient_needs_neither_operand():
    dy = randn((ROWS, N), 1).to(DEV)
    x8, w8 = dg.fp8_quantize(randn((ROWS, K), 2).to(DEV)), dg.fp8_quantize(randn((N, K), 3).to(DEV), 128)
    every = dg.fp8_linear_backward(x8, w8, dy, need_db=True)["bias"]
    assert torch.equal(dg.fp8_linear_backward(None, None, dy, False, False, True)["bias"], every)
    for need in ((True, False), (False, True)):
        with pytest.raises(ValueError):
            dg.fp8_linear_backward(None, None, dy, *need, True)

"""The bf16 layers that keep 8-bit activations quantise them only where a backward will read them."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from test_gpu_fp8 import DEV, randn

pytestmark = pytest.mark.gpu


def quantised(call):
    """(result, launches of the quantiser)"""
    dg.trace_begin("fp8_quantize")
    try:
        y = call()
    finally:
        seen = dg.trace_end()
    return y, sum(t["launches"] for t in seen)


def linear():
    x, w, b = randn((2, 33, 144), 1).to(DEV), randn((176, 144), 2, 0.1).to(DEV), randn((176,), 3).to(DEV)
    return dg.tp_linear_layer_keep8, dg.tp_linear(x, w, b), [x, w, b]


def swiglu():
    x, w13, w2 = (randn(s, i, 0.2).to(DEV) for i, s in enumerate(((2, 1, 16, 64), (2, 64, 64), (64, 64))))
    return dg.tp_swiglu_layer_keep8, dg.tp_swiglu(x, w13, w2), [x, w13, w2]


@pytest.mark.parametrize("make", [linear, swiglu])
def test_nothing_is_quantised_where_nothing_is_recorded(make):
    layer, y, args = make()
    got, n = quantised(lambda: layer(*args))   # nothing requires a gradient
    assert torch.equal(got, y) and n == 0 and not got.requires_grad
    for t in args:
        t.requires_grad_()
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            got, n = quantised(lambda: layer(*args))
        assert torch.equal(got, y) and n == 0 and not got.requires_grad
    got, n = quantised(lambda: layer(*args))
    assert torch.equal(got.detach(), y) and n == 1 and got.requires_grad


@pytest.mark.parametrize("make", [linear, swiglu])
@pytest.mark.parametrize("trained", [(0,), (1,), (2,), (0, 2), (1, 2)])
def test_some_inputs_trained(make, trained):
    layer, y, args = make()
    for t in args:
        t.requires_grad_()
    dy = randn(tuple(y.shape), 9).to(DEV)
    every = torch.autograd.grad(layer(*args), args, dy)
    for i, t in enumerate(args):
        t.requires_grad_(i in trained)
    got, n = quantised(lambda: layer(*args))
    assert torch.equal(got.detach(), y) and n == (1 if make is swiglu or 1 in trained else 0)
    for i, g in zip(trained, torch.autograd.grad(got, [args[i] for i in trained], dy)):
        assert torch.equal(g, every[i])


@pytest.mark.parametrize("make", [linear, swiglu])
def test_forward_mode_is_refused(make):
    """Forward derivatives are not defined: an error, also where nothing is recorded for a backward."""
    layer, _, args = make()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(args[0], torch.ones_like(args[0]))
        for on in (True, False):
            with torch.set_grad_enabled(on), pytest.raises(RuntimeError):
                layer(dual, *args[1:])


def test_the_functions_take_their_inputs_alone():
    """TPLinearKeep8 and TPSwiGLUKeep8 are public: called without the layers they keep what a backward reads."""
    for make, fn in ((linear, dg.TPLinearKeep8), (swiglu, dg.TPSwiGLUKeep8)):
        layer, y, args = make()
        for t in args:
            t.requires_grad_()
        dy = randn(tuple(y.shape), 9).to(DEV)
        a, b = (torch.autograd.grad(f(*args), args, dy) for f in (layer, fn.apply))
        assert all(torch.equal(p, q) for p, q in zip(a, b))

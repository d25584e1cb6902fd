"""tp_linear's backward with a frozen weight reads no x, so it asks for none."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from test_fp8_refusals import INVALID, lib, mem  # noqa: F401  (fixtures)

BF16 = torch.bfloat16


def test_x_may_be_null_without_the_weight_gradient(lib, mem):
    x, w, dy, dx, dw, db, ws = mem[:7]

    def call(x, dx, dw, db, ws, n):
        return lib.dg_tp_linear_bwd(2, 64, 16, x, w, dy, dx, dw, db, ws, n, None)

    for x_, out in ((None, (dx, dw, db)), (None, (None, dw, None))):
        assert call(x_, *out, ws, 256) == INVALID and b"x is NULL" in lib.dg_last_error()
    for out in ((dx, None, None), (dx, None, db), (None, None, db)):
        st = call(None, *out, None, 0)                       # refused for its workspace, not for x
        assert st != 0 and b"x is NULL" not in lib.dg_last_error()
    assert call(None, dy, None, None, ws, 256) == INVALID and b"overlap" in lib.dg_last_error()


def test_refusals_before_the_device():
    w, dy = torch.zeros(16, 64, dtype=BF16), torch.zeros(2, 16, dtype=BF16)
    with pytest.raises(ValueError, match="x is needed"):
        dg.tp_linear_backward(None, w, dy)
    with pytest.raises(ValueError, match="CUDA"):
        dg.tp_linear_backward(None, w, dy, need_dw=False)
    with pytest.raises(TypeError):
        dg.tp_linear_backward(None, w, None, need_dw=False)


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [(1,), (70,), (2, 33)])
def test_gradients_without_x(lead):
    from test_gpu_fp8 import DEV, randn
    x, w, dy = randn((*lead, 144), 1).to(DEV), randn((176, 144), 2, 0.1).to(DEV), randn((*lead, 176), 3).to(DEV)
    every = dg.tp_linear_backward(x, w, dy, need_db=True)
    g = dg.tp_linear_backward(None, w, dy, need_dw=False, need_db=True)
    assert torch.equal(g["x"], every["x"]) and torch.equal(g["bias"], every["bias"]) and g["weight"] is None
    with pytest.raises(ValueError):
        dg.tp_linear_backward(None, w, dy[..., :168].contiguous(), need_dw=False)
    with pytest.raises(TypeError):
        dg.tp_linear_backward(None, w, dy.float(), need_dw=False)


@pytest.mark.gpu
def test_memory_of_the_backward_with_a_frozen_weight():
    """keep8 with a frozen weight: its backward allocates the input's gradient, and no second tensor of that size."""
    from test_gpu_fp8 import DEV, randn
    x, w = randn((4096, 8192), 1).to(DEV).requires_grad_(), randn((256, 8192), 2, 0.01).to(DEV)
    dy = randn((4096, 256), 3).to(DEV)
    y = dg.tp_linear_layer_keep8(x, w)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    (g,) = torch.autograd.grad(y, (x,), dy)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= g.numel() * 2 + (4 << 20)

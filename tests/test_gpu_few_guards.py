"""Guard regions around every buffer the few-token operators write: outputs
and workspaces sit between sentinel bytes that must survive the call."""
import ctypes

import pytest
import torch

import expert_gemm_layers_gb300 as dg
from expert_gemm_layers_gb300 import _lib
from test_gpu_few import BF16, DEV, randn, routing, w4_weight
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,K,group", [(1, 32, 32), (13, 96, 32), (5, 192, 64), (33, 128, 128)])
@pytest.mark.parametrize("zero_points", [False, True])
def test_w4_quantize_and_dequantize_write_only_their_outputs(rows, K, group, zero_points):
    lib, g = _lib.load(), Guarded()
    w = randn((rows, K), rows).to(DEV)
    codes, scales = g.raw(rows * K // 2), g.tensor((rows, K // group), BF16)
    zeros = g.raw(rows * K // group) if zero_points else None
    back = g.tensor((rows, K), BF16)
    s = torch.cuda.current_stream().cuda_stream
    p = lambda t: None if t is None else t.data_ptr()
    _lib.check(lib.dg_w4_quantize(rows, K, group, p(w), p(codes), p(scales), p(zeros), s))
    _lib.check(lib.dg_w4_dequantize(rows, K, group, p(codes), p(scales), p(zeros), p(back), s))
    g.check(f"w4 {rows, K, group}")
    assert torch.isfinite(back.float()).all()


@pytest.mark.parametrize("rows,K,N,group", [(1, 64, 1, 32), (9, 256, 17, 64), (35, 128, 130, 128)])
def test_w4_linear_writes_only_y(rows, K, N, group):
    g = Guarded()
    w, _ = w4_weight((), N, K, group, True, 1)
    y = g.tensor((rows, N), BF16)
    need = _lib.load().dg_w4_linear_workspace_bytes(rows, K, N)
    dg.w4_linear(randn((rows, K), 2).to(DEV), *w, out=y, ws=g.workspace(need))
    g.check(f"w4_linear {rows, K, N, group}")
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("T,d,E,k", [(1, 64, 5, 2), (7, 72, 70, 9)])
def test_moe_route_writes_only_its_outputs(T, d, E, k):
    lib, g = _lib.load(), Guarded()
    x, w = randn((T, d), 1).to(DEV), randn((E, d), 2).to(DEV)
    idx, gates = g.tensor((T, k), torch.int32), g.tensor((T, k), torch.float32)
    ws = g.workspace(lib.dg_moe_route_workspace_bytes(T, d, E, k))
    _lib.check(lib.dg_moe_route(T, d, E, k, 2, 1.0, x.data_ptr(), w.data_ptr(), idx.data_ptr(), gates.data_ptr(),
                                ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
    g.check(f"moe_route {T, d, E, k}")
    assert torch.all((idx >= 0) & (idx < E))


@pytest.mark.parametrize("T,d,F,E,k,group", [(1, 72, 40, 3, 2, 0), (19, 136, 8, 4, 3, 0), (3, 128, 96, 4, 2, 32),
                                             (40, 64, 192, 2, 2, 64)])
def test_moe_swiglu_writes_only_y_and_its_workspace(T, d, F, E, k, group):
    lib, g = _lib.load(), Guarded()
    idx, gates = (t.to(DEV) for t in routing(T, E, k, 3))
    x = randn((T, d), 1).to(DEV)
    sh = _lib.MoEShape(T, d, F, E, k)
    ws = g.workspace(lib.dg_moe_swiglu_workspace_bytes(ctypes.byref(sh), group))
    y = g.tensor((T, d), BF16)
    if group:
        w13, w2 = w4_weight((E,), 2 * F, d, group, True, 4)[0], w4_weight((E,), d, F, group, True, 5)[0]
        dg.moe_swiglu_w4(x, idx, gates, w13, w2, workspace=ws, out=y)
    else:
        dg.moe_swiglu(x, idx, gates, randn((E, 2 * F, d), 4, 0.1).to(DEV), randn((E, d, F), 5, 0.1).to(DEV),
                      workspace=ws, out=y)
    g.check(f"moe_swiglu {T, d, F, E, k, group}")
    assert torch.isfinite(y.float()).all()

"""Block-scaled e4m3 operators and the memory around their buffers: outputs and workspaces sit between sentinel bytes
that must survive the call, and a workspace that holds a recorded failure keeps its calls from writing."""
import pytest
import torch

import expert_gemm_layers_gb300 as dg
from expert_gemm_layers_gb300 import _lib, alloc_workspace, debug_wait_timeout, device_status
from test_gpu_fp8 import BF16, DEV, E4M3, E8M0, randn
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu
DG_ERR_TIMEOUT = 4


def stream():
    return torch.cuda.current_stream().cuda_stream


def p(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("rows,K", [(1, 16), (13, 144), (130, 272), (257, 400), (4100, 2064)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_and_dequantize(rows, K, block_rows):
    lib, g = _lib.load(), Guarded()
    x = randn((rows, K), rows).to(DEV)
    codes = g.tensor((rows, K), E4M3)
    scales = g.tensor((-(-rows // block_rows), -(-K // 128)), E8M0)
    back = g.tensor((rows, K), BF16)
    _lib.check(lib.dg_fp8_quantize(rows, K, block_rows, p(x), p(codes), p(scales), stream()))
    _lib.check(lib.dg_fp8_dequantize(rows, K, block_rows, p(codes), p(scales), p(back), stream()))
    g.check(f"quantize {rows, K, block_rows}")
    assert torch.isfinite(back.float()).all()


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (7, 272, 144), (33, 528, 240), (65, 144, 464), (100, 8208, 272), (300, 400, 688)])
@pytest.mark.parametrize("bf16", [False, True])
def test_linear(rows, K, N, bf16):
    lib, g = _lib.load(), Guarded()
    x = randn((rows, K), 1).to(DEV)
    w8 = dg.fp8_quantize(randn((N, K), 2).to(DEV), 128)
    need = (lib.dg_fp8_linear_bf16_workspace_bytes if bf16 else lib.dg_fp8_linear_workspace_bytes)(rows, K, N)
    y = g.tensor((rows, N), BF16)
    dg.fp8_linear(x if bf16 else dg.fp8_quantize(x), w8, randn((N,), 3).to(DEV), out=y, workspace=g.workspace(need))
    g.check(f"fp8_linear {rows, K, N}")
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("rows,K,N", [(1, 16, 16), (33, 272, 144), (300, 400, 688), (2060, 144, 272)])
def test_linear_backward(rows, K, N):
    lib, g = _lib.load(), Guarded()
    xc, xs = dg.fp8_quantize(randn((rows, K), 1).to(DEV))
    wc, wscale = dg.fp8_quantize(randn((N, K), 2).to(DEV), 128)
    dy = randn((rows, N), 3).to(DEV)
    dx, dw, db = g.tensor((rows, K), BF16), g.tensor((N, K), BF16), g.tensor((N,), BF16)
    ws = g.workspace(lib.dg_fp8_linear_bwd_workspace_bytes(rows, K, N))
    _lib.check(lib.dg_fp8_linear_bwd(rows, K, N, p(xc), p(xs), p(wc), p(wscale), p(dy), p(dx), p(dw), p(db), p(ws),
                                     lib.dg_fp8_linear_bwd_workspace_bytes(rows, K, N), stream()))
    g.check(f"fp8_linear_bwd {rows, K, N}")
    assert all(torch.isfinite(t.float()).all() for t in (dx, dw, db))


@pytest.mark.parametrize("rows,d", [(1, 8), (5, 136), (9, 520), (33, 1288), (7, 4104), (3, 8200), (2, 16400)])
def test_norm(rows, d):
    lib, g = _lib.load(), Guarded()
    x, r, w, dy = (randn(s, i).to(DEV) for i, s in enumerate(((rows, d), (rows, d), (d,), (rows, d))))
    h, y, dx, dw = g.tensor((rows, d), BF16), g.tensor((rows, d), BF16), g.tensor((rows, d), BF16), g.tensor((d,), BF16)
    _lib.check(lib.dg_rms_norm(rows, d, 1e-6, p(x), p(r), p(w), p(h), p(y), None, None, stream()))
    need = lib.dg_rms_norm_bwd_workspace_bytes(rows, d)
    ws = g.workspace(need)
    _lib.check(lib.dg_rms_norm_bwd(rows, d, 1e-6, p(h), p(w), p(dy), p(r), p(dx), p(dw), p(ws), need, stream()))
    if d % 16 == 0:
        codes, scales = g.tensor((rows, d), E4M3), g.tensor((rows, -(-d // 128)), E8M0)
        _lib.check(lib.dg_rms_norm(rows, d, 1e-6, p(x), p(r), p(w), p(h), None, p(codes), p(scales), stream()))
    g.check(f"rms_norm {rows, d}")
    assert all(torch.isfinite(t.float()).all() for t in (h, y, dx, dw))


def test_nothing_is_written_after_a_recorded_failure():
    lib = _lib.load()
    for rows in (3, 100, 2060):
        x, w8 = randn((rows, 272), 1).to(DEV), dg.fp8_quantize(randn((400, 272), 2).to(DEV), 128)
        x8, dy = dg.fp8_quantize(x), randn((rows, 400), 3).to(DEV)
        need = max(lib.dg_fp8_linear_bwd_workspace_bytes(rows, 272, 400), lib.dg_fp8_linear_bf16_workspace_bytes(rows, 272, 400),
                   lib.dg_rms_norm_bwd_workspace_bytes(rows, 272))
        ws = alloc_workspace(need, DEV)
        outs = [torch.full(s, 7.0, dtype=BF16, device=DEV) for s in ((rows, 400), (rows, 272), (400, 272), (400,), (rows, 272), (272,))]
        y, dx, dw, db, nx, nw = outs

        def calls():
            dg.fp8_linear(x, w8, out=y, workspace=ws)
            dg.fp8_linear(x8, w8, out=y, workspace=ws)
            _lib.check(lib.dg_fp8_linear_bwd(rows, 272, 400, p(x8[0]), p(x8[1]), p(w8[0]), p(w8[1]), p(dy), p(dx), p(dw),
                                             p(db), p(ws), ws.numel(), stream()))
            _lib.check(lib.dg_rms_norm_bwd(rows, 272, 1e-6, p(x), p(x[0]), p(x), None, p(nx), p(nw), p(ws), ws.numel(),
                                           stream()))

        debug_wait_timeout(10_000, workspace=ws)
        calls()
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in outs)
        assert device_status(workspace=ws)[0] == DG_ERR_TIMEOUT
        calls()
        torch.cuda.synchronize()
        assert all(not (t == 7).all() for t in outs)
        assert device_status(workspace=ws)[0] == 0

"""Refusals of the few-token operators, without a GPU: the C entry points
reject bad arguments before any device call, the wrappers before that."""
import ctypes
import os

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    from expert_gemm_layers_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from expert_gemm_layers_gb300 import build
        build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def mem():
    """Twelve 64 KiB regions standing in for device tensors (never dereferenced)."""
    buf = ctypes.create_string_buffer(13 << 16)
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    yield [base + (i << 16) for i in range(12)]
    del buf


def test_w4_quantize_and_dequantize(lib, mem):
    w, c, s, z = mem[:4]
    for call, what in ((lambda *a: lib.dg_w4_quantize(*a[:3], w, *a[3:], None), "w4_quantize"),
                       (lambda *a: lib.dg_w4_dequantize(*a[:3], *a[3:], w, None), "w4_dequantize")):
        assert call(4, 128, 16, c, s, z) == INVALID and b"group" in lib.dg_last_error()
        assert call(4, 130, 32, c, s, z) == INVALID and b"multiple" in lib.dg_last_error()
        assert call(-1, 128, 32, c, s, z) == INVALID
        assert call(4, 0, 32, c, s, z) == INVALID
        assert call(1 << 31, 1 << 20, 32, c, s, z) == UNSUPPORTED
        assert call(4, 128, 32, None, s, z) == INVALID and b"codes is NULL" in lib.dg_last_error()
        assert call(4, 128, 32, c, s + 8, z) == INVALID and b"aligned" in lib.dg_last_error()
        assert call(0, 128, 32, None, None, None) == OK            # no rows: nothing to do
        assert what.encode() not in b"" and call(4, 128, 32, w, s, z) == INVALID and b"overlaps" in lib.dg_last_error()


def test_w4_linear(lib, mem):
    x, c, s, z, b, y, ws = mem[:7]
    ok = dict(rows=2, K=128, N=16, g=32, x=x, c=c, s=s, z=z, b=b, y=y, ws=ws, n=256)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_w4_linear(a["rows"], a["K"], a["N"], a["g"], a["x"], a["c"], a["s"], a["z"], a["b"], a["y"],
                                a["ws"], a["n"], None)

    assert call(rows=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(g=48) == INVALID and call(K=144) == INVALID
    assert call(rows=65535 * 32 + 1) == UNSUPPORTED
    assert call(N=(1 << 31) - 100, K=32) == UNSUPPORTED
    assert call(x=None) == INVALID and call(s=None) == INVALID and call(y=None) == INVALID
    assert call(y=x) == INVALID and call(y=ws) == INVALID and b"overlaps" in lib.dg_last_error()
    assert call(ws=None) == WORKSPACE and call(n=128) == WORKSPACE and call(ws=ws + 8) == INVALID
    assert call(rows=0, x=None, y=None, ws=None) == OK


def test_moe_route(lib, mem):
    x, w, i, gt, ws = mem[:5]
    ok = dict(T=2, d=64, E=8, k=2, f=0, x=x, w=w, i=i, g=gt, ws=ws, n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_moe_route(a["T"], a["d"], a["E"], a["k"], a["f"], 1.0, a["x"], a["w"], a["i"], a["g"], a["ws"],
                                a["n"], None)

    assert call(T=-1) == INVALID and call(d=63) == INVALID and call(E=0) == INVALID
    assert call(k=0) == INVALID and call(k=9) == INVALID and call(f=4) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(E=64, k=33) == UNSUPPORTED and call(T=65535 * 4 + 1) == UNSUPPORTED
    assert call(i=None) == INVALID and call(g=gt + 4) == INVALID and call(g=i) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE
    assert call(T=0, x=None, w=None, i=None, g=None, ws=None) == OK


def test_moe_swiglu(lib, mem):
    from expert_gemm_layers_gb300._lib import MoEShape
    x, i, gt, w13, w2, y, ws = mem[:7]
    ok = dict(T=2, d=64, F=32, E=4, k=2, x=x, i=i, g=gt, a=w13, b=w2, y=y, ws=ws, n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        sh = MoEShape(a["T"], a["d"], a["F"], a["E"], a["k"])
        return lib.dg_moe_swiglu(ctypes.byref(sh), a["x"], a["i"], a["g"], a["a"], a["b"], a["y"], a["ws"], a["n"],
                                 None)

    assert lib.dg_moe_swiglu(None, *([None] * 7), 0, None) == INVALID
    assert call(T=-1) == INVALID and call(d=60) == INVALID and call(F=4) == INVALID and call(E=0) == INVALID
    assert call(k=0) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(k=33) == UNSUPPORTED and call(d=(1 << 20) + 8) == UNSUPPORTED
    assert call(T=4097, k=2) == UNSUPPORTED and b"split" in lib.dg_last_error()
    assert call(x=None) == INVALID and call(b=None) == INVALID and call(y=x) == INVALID and call(y=w13) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=256) == WORKSPACE
    assert call(T=0, x=None, i=None, g=None, a=None, b=None, y=None, ws=None) == OK
    sh = MoEShape(2, 64, 32, 4, 2)
    for group in (0, 32):
        assert lib.dg_moe_swiglu_workspace_bytes(ctypes.byref(sh), group) >= 256 + 4 * 32 * 2 + 4 * 64 * 4
    assert lib.dg_moe_swiglu_workspace_bytes(ctypes.byref(sh), 16) == 0
    sh = MoEShape(2, 60, 32, 4, 2)
    assert lib.dg_moe_swiglu_workspace_bytes(ctypes.byref(sh), 0) == 0


def test_moe_swiglu_w4(lib, mem):
    from expert_gemm_layers_gb300._lib import MoEShape
    p = mem
    ok = dict(T=2, d=64, F=32, E=4, k=2, grp=32, z13=p[5], z2=p[8])

    def call(**kw):
        a = {**ok, **kw}
        sh = MoEShape(a["T"], a["d"], a["F"], a["E"], a["k"])
        return lib.dg_moe_swiglu_w4(ctypes.byref(sh), a["grp"], p[0], p[1], p[2], p[3], p[4], a["z13"], p[6], p[7],
                                    a["z2"], a.get("y", p[9]), a.get("ws", p[10]), 1 << 16, None)

    assert call(grp=64) == INVALID and call(grp=16) == INVALID and call(F=40) == INVALID
    assert call(z2=None) == INVALID and b"zeros" in lib.dg_last_error()
    assert call(ws=None) == WORKSPACE and call(y=p[7]) == INVALID
    assert call(T=0) == OK


def test_wrappers_refuse_before_the_device():
    import expert_gemm_layers_gb300 as dg
    bf = torch.bfloat16
    x = torch.zeros(2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        dg.w4_quantize(x, 32)
    with pytest.raises(TypeError):
        dg.w4_quantize(x.float(), 32)
    with pytest.raises(ValueError, match="CUDA"):
        dg.moe_route(x, x, 1)
    with pytest.raises(ValueError, match="score"):
        dg.moe_route(x, x, 1, score="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        dg.w4_linear(x, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        dg.moe_swiglu(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(1, 16, 64, dtype=bf),
                      torch.zeros(1, 64, 8, dtype=bf))

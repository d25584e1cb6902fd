"""Refusals of the block-scaled e4m3 operators, without a GPU: the C entry points
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


def test_quantize_and_dequantize(lib, mem):
    x, c, s = mem[:3]
    for call in (lambda r, K, b, x, c, s: lib.dg_fp8_quantize(r, K, b, x, c, s, None),
                 lambda r, K, b, x, c, s: lib.dg_fp8_dequantize(r, K, b, c, s, x, None)):
        assert call(4, 128, 2, x, c, s) == INVALID and b"block_rows" in lib.dg_last_error()
        assert call(4, 120, 1, x, c, s) == INVALID and b"multiple of 16" in lib.dg_last_error()
        assert call(-1, 128, 1, x, c, s) == INVALID and call(4, 0, 1, x, c, s) == INVALID
        assert call(1 << 31, 128, 1, x, c, s) == UNSUPPORTED and call(1 << 30, 2048, 1, x, c, s) == UNSUPPORTED
        assert call(4, 128, 1, None, c, s) == INVALID and call(4, 128, 1, x, c + 8, s) == INVALID
        assert call(4, 128, 1, x, c, None) == INVALID and b"scales is NULL" in lib.dg_last_error()
        assert call(4, 128, 1, x, x, s) == INVALID and b"overlaps" in lib.dg_last_error()
        assert call(0, 128, 128, None, None, None) == OK


def test_linear(lib, mem):
    ok = dict(rows=2, K=128, N=16, xc=mem[0], xs=mem[1], wc=mem[2], ws=mem[3], b=mem[4], y=mem[5], w=mem[6], n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_fp8_linear(*(a[k] for k in ("rows", "K", "N", "xc", "xs", "wc", "ws", "b", "y", "w", "n")), None)

    assert call(rows=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(K=136) == INVALID and call(N=24) == INVALID and b"multiples of 16" in lib.dg_last_error()
    assert call(N=(1 << 31) - 1024, K=16) == UNSUPPORTED and call(rows=(1 << 31) - 1024) == UNSUPPORTED
    for name in ("xc", "xs", "wc", "ws", "y"):
        assert call(**{name: None}) == INVALID
    for name in ("xc", "wc", "y", "b"):
        assert call(**{name: ok[name] + 4}) == INVALID and b"aligned" in lib.dg_last_error()
    assert call(y=ok["xc"]) == INVALID and call(y=ok["w"]) == INVALID and call(b=ok["y"]) == INVALID
    assert call(w=None) == WORKSPACE and call(n=255) == WORKSPACE
    assert call(rows=0, xc=None, xs=None, wc=None, ws=None, b=None, y=None, w=None) == OK
    assert lib.dg_fp8_linear_workspace_bytes(2, 136, 16) == 0 and lib.dg_fp8_linear_workspace_bytes(2, 128, 16) >= 256


def test_linear_bf16(lib, mem):
    ok = dict(rows=2, K=128, N=16, x=mem[0], wc=mem[2], ws=mem[3], b=mem[4], y=mem[5], w=mem[6], n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_fp8_linear_bf16(*(a[k] for k in ("rows", "K", "N", "x", "wc", "ws", "b", "y", "w", "n")), None)

    assert call(rows=-1) == INVALID and call(K=136) == INVALID and call(N=24) == INVALID
    for name in ("x", "wc", "ws", "y"):
        assert call(**{name: None}) == INVALID and b"NULL" in lib.dg_last_error()
    assert call(y=ok["x"]) == INVALID and call(y=ok["w"]) == INVALID and call(w=None) == WORKSPACE
    need = lib.dg_fp8_linear_bf16_workspace_bytes(2, 128, 16)
    assert need >= 256 + 2 * 128 + 2 and call(n=need - 1) == WORKSPACE
    assert lib.dg_fp8_linear_bf16_workspace_bytes(2, 136, 16) == 0
    assert call(rows=0, x=None, wc=None, ws=None, b=None, y=None, w=None) == OK


def test_linear_bwd(lib, mem):
    ok = dict(rows=2, K=128, N=16, xc=mem[0], xs=mem[1], wc=mem[2], ws=mem[3], dy=mem[4], dx=mem[5], dw=mem[6],
              db=mem[7], w=mem[8], n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_fp8_linear_bwd(*(a[k] for k in ("rows", "K", "N", "xc", "xs", "wc", "ws", "dy", "dx", "dw", "db",
                                                      "w", "n")), None)

    assert call(rows=-1) == INVALID and call(K=8) == INVALID and call(N=8) == INVALID
    for name in ("xc", "xs", "wc", "ws", "dy"):
        assert call(**{name: None}) == INVALID and b"NULL" in lib.dg_last_error()
    assert call(dx=ok["dw"]) == INVALID and call(db=ok["dy"]) == INVALID and call(dw=ok["w"]) == INVALID
    assert call(w=None) == WORKSPACE
    need = lib.dg_fp8_linear_bwd_workspace_bytes(2, 128, 16)
    assert need >= 256 + 2 * 16 + 2 + 2 * 2 * 128 and call(n=need - 1) == WORKSPACE
    assert lib.dg_fp8_linear_bwd_workspace_bytes(2, 100, 16) == 0


def test_rms_norm(lib, mem):
    ok = dict(rows=2, d=64, eps=1e-6, x=mem[0], r=mem[1], w=mem[2], h=mem[3], y=mem[4], c=None, s=None)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_rms_norm(*(a[k] for k in ("rows", "d", "eps", "x", "r", "w", "h", "y", "c", "s")), None)

    assert call(rows=-1) == INVALID and call(d=0) == INVALID and call(d=60) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(d=32776) == UNSUPPORTED and call(rows=1 << 31) == UNSUPPORTED
    assert call(x=None) == INVALID and call(w=None) == INVALID and call(r=None) == INVALID and call(h=None) == INVALID
    assert call(y=None) == INVALID and call(c=mem[5]) == INVALID and call(c=mem[5], s=mem[6]) == INVALID
    assert call(y=None, c=mem[5], s=mem[6], d=72) == INVALID and b"16" in lib.dg_last_error()
    assert call(h=ok["r"]) == INVALID and call(y=ok["x"]) == INVALID and call(y=ok["h"]) == INVALID
    assert call(x=mem[0] + 2) == INVALID and b"aligned" in lib.dg_last_error()
    assert call(rows=0, x=None, r=None, w=None, h=None, y=None) == OK


def test_rms_norm_bwd(lib, mem):
    ok = dict(rows=2, d=64, eps=1e-6, h=mem[0], w=mem[1], dy=mem[2], dh=mem[3], dx=mem[4], dw=mem[5], ws=mem[6], n=1 << 16)

    def call(**kw):
        a = {**ok, **kw}
        return lib.dg_rms_norm_bwd(*(a[k] for k in ("rows", "d", "eps", "h", "w", "dy", "dh", "dx", "dw", "ws", "n")), None)

    assert call(rows=-1) == INVALID and call(d=12) == INVALID and call(eps=-1.0) == INVALID
    assert call(h=None) == INVALID and call(dy=None) == INVALID and call(w=None) == INVALID
    assert call(dx=ok["dy"]) == INVALID and call(dw=ok["w"]) == INVALID and call(dx=ok["ws"]) == INVALID
    need = lib.dg_rms_norm_bwd_workspace_bytes(2, 64)
    assert need > 256 and call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert lib.dg_rms_norm_bwd_workspace_bytes(2, 60) == 0


def test_wrappers_refuse_before_the_device():
    import expert_gemm_layers_gb300 as dg
    bf = torch.bfloat16
    x, pair = torch.zeros(2, 64, dtype=bf), (torch.zeros(2, 64).to(torch.float8_e4m3fn), torch.ones(2, 1).to(torch.float8_e8m0fnu))
    for call in (lambda: dg.fp8_quantize(x), lambda: dg.fp8_dequantize(*pair), lambda: dg.fp8_linear(x, pair),
                 lambda: dg.fp8_linear(pair, pair), lambda: dg.fp8_linear_backward(pair, pair, x), lambda: dg.rms_norm(x, x[0]),
                 lambda: dg.rms_norm_backward(x, x[0], x), lambda: dg.fp8_linear_layer(x, x),
                 lambda: dg.tp_linear_layer_keep8(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        dg.fp8_quantize(x.float())
    for other in (None, 3, "x"):
        with pytest.raises(TypeError):
            dg.fp8_quantize(other)
        with pytest.raises(TypeError):
            dg.rms_norm(other, x)
        with pytest.raises(TypeError):
            dg.fp8_linear(other, pair)
    with pytest.raises(TypeError):
        dg.fp8_linear(pair[0], pair)
    with pytest.raises(TypeError, match="codes, scales"):
        dg.fp8_linear((pair[0],), pair)

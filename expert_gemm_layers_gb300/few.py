"""Torch-facing wrappers of the few-token operators: 4-bit weights and routed experts.

As in ops.py, each function checks its arguments, allocates outputs and
scratch with torch and passes pointers and the current stream to the C ABI.
Weights in 4 bits are (codes, scales, zeros) as w4_quantize returns them:
codes [..., K/2] uint8, scales [..., K/group] bf16, zeros [..., K/group] uint8
or None (zero point 8).  None of these operators has a backward: inputs that
require gradients are taken as constants.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import DG_ERROR_BLOCK_BYTES, DG_MOE_RENORM, DG_MOE_SIGMOID, MoEShape, check, load
from .ops import _need, _stream, alloc_workspace, error_block

__all__ = ["w4_quantize", "w4_dequantize", "w4_linear", "moe_route", "moe_swiglu", "moe_swiglu_w4", "moe_layer"]


def _launch(fn, dev: torch.device, *args) -> None:
    """fn(*args, stream) with `dev` current."""
    if torch.cuda.current_device() == dev.index:
        check(fn(*args, _stream(dev)))
    else:
        with torch.cuda.device(dev):
            check(fn(*args, _stream(dev)))


def _p(t):
    return None if t is None else t.data_ptr()


_scratch_cache: dict = {}


def _scratch(dev: torch.device, nbytes: int) -> torch.Tensor:
    """The workspace this module gives calls that bring none: one per (device,
    current stream), grown as needed, its error block zeroed when it is made.
    A captured call gets one of its own, in the graph's memory, so that graphs
    captured on one stream do not share it."""
    if nbytes <= DG_ERROR_BLOCK_BYTES:
        return error_block(dev)
    if torch.cuda.is_current_stream_capturing():
        return alloc_workspace(nbytes, dev)
    key = (dev.index, _stream(dev))
    ws = _scratch_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _scratch_cache[key] = alloc_workspace(nbytes, dev)
    return ws


def _need_workspace(ws: torch.Tensor, nbytes: int, dev: torch.device) -> None:
    _need(ws, "workspace", torch.uint8, None, dev)
    if ws.numel() < nbytes:
        raise ValueError(f"workspace has {ws.numel()} bytes, needs {nbytes}")


# ------------------------------------------------------------------ 4-bit weights

def _need_w4(codes, scales, zeros, lead: tuple, K: int, dev, what: str) -> int:
    """Checks one 4-bit weight [*lead, K]; returns its group size."""
    _need(codes, f"{what}codes", torch.uint8, (*lead, K // 2), dev)
    if not isinstance(scales, torch.Tensor) or scales.dim() != codes.dim() or scales.shape[-1] < 1 \
            or K % scales.shape[-1]:
        raise ValueError(f"{what}scales must be [..., K/group] beside codes [..., K/2]")
    _need(scales, f"{what}scales", torch.bfloat16, (*lead, scales.shape[-1]), dev)
    if zeros is not None:
        _need(zeros, f"{what}zeros", torch.uint8, scales.shape, dev)
    return K // scales.shape[-1]


def w4_quantize(weight: torch.Tensor, group: int = 128, zero_points: bool = False):
    """4-bit codes of a bf16 weight [..., K] with one scale per `group` columns (32, 64 or 128).

    Returns (codes, scales, zeros): value = (code - zero) * scale.  zeros is
    None unless zero_points (then codes span each group's own range instead of
    a symmetric one)."""
    lib = load()
    _need(weight, "weight", torch.bfloat16)
    K = weight.shape[-1]
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide {K}, got {group}")
    lead, dev = weight.shape[:-1], weight.device
    codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((*lead, K // group), dtype=torch.bfloat16, device=dev)
    zeros = torch.empty((*lead, K // group), dtype=torch.uint8, device=dev) if zero_points else None
    rows = weight.numel() // K if K else 0
    _launch(lib.dg_w4_quantize, dev, rows, K, group, _p(weight), _p(codes), _p(scales), _p(zeros))
    return codes, scales, zeros


def w4_dequantize(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 weight [..., K] that 4-bit codes stand for."""
    lib = load()
    _need(codes, "codes", torch.uint8)
    K, lead, dev = 2 * codes.shape[-1], codes.shape[:-1], codes.device
    group = _need_w4(codes, scales, zeros, tuple(lead), K, dev, "")
    if out is None:
        out = torch.empty((*lead, K), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (*lead, K), dev)
    _launch(lib.dg_w4_dequantize, dev, out.numel() // K if K else 0, K, group, _p(codes), _p(scales), _p(zeros), _p(out))
    return out


def w4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W^T (+ bias) with W [out, in] in 4 bits, for few rows x [..., in] (a decode step).

    Sums in binary32, one rounding to bf16.  For long prompts dequantise once
    and use tp_linear.  `ws` holds the call's error block (default: this
    stream's own), and scratch where there are more than few short rows
    (dg_w4_linear_workspace_bytes)."""
    lib = load()
    in_f, dev = x.shape[-1], x.device
    _need(x, "x", torch.bfloat16)
    out_f = codes.shape[0]
    group = _need_w4(codes, scales, zeros, (out_f,), in_f, dev, "")
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, (out_f,), dev)
    if out is None:
        out = torch.empty((*x.shape[:-1], out_f), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, (*x.shape[:-1], out_f), dev)
    rows = x.numel() // in_f if in_f else 0
    if ws is None:
        ws = _scratch(dev, lib.dg_w4_linear_workspace_bytes(rows, in_f, out_f))
    _launch(lib.dg_w4_linear, dev, rows, in_f, out_f, group, _p(x), _p(codes), _p(scales), _p(zeros),
            _p(bias), _p(out), _p(ws), ws.numel())
    return out


# ------------------------------------------------------------------ routed experts

def moe_route(x: torch.Tensor, w_router: torch.Tensor, top_k: int, score: str = "softmax", renormalize: bool = True,
              scale: float = 1.0, workspace: torch.Tensor | None = None):
    """The top_k experts of each token and their gates.

    x [T, d], w_router [E, d] bf16; logits x @ w_router^T are rounded once to
    binary32, equal logits go to the lower expert.  score: "softmax" or
    "sigmoid"; renormalize divides the gates by their sum over the chosen
    experts (softmax otherwise: over all experts); scale multiplies them.
    Returns idx [T, top_k] int32 (largest logit first) and gates [T, top_k]
    binary32."""
    lib = load()
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    _need(x, "x", torch.bfloat16)
    T, d = x.shape
    E, dev = w_router.shape[0], x.device
    _need(w_router, "w_router", torch.bfloat16, (E, d), dev)
    flags = (DG_MOE_SIGMOID if score == "sigmoid" else 0) | (DG_MOE_RENORM if renormalize else 0)
    idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    nbytes = lib.dg_moe_route_workspace_bytes(T, d, E, top_k)
    if workspace is None:
        workspace = _scratch(dev, nbytes)
    else:
        _need_workspace(workspace, nbytes, dev)
    _launch(lib.dg_moe_route, dev, T, d, E, top_k, flags, float(scale), _p(x), _p(w_router), _p(idx), _p(gates),
            _p(workspace), workspace.numel())
    return idx, gates


def _moe_args(x, idx, gates, workspace, out, F: int, E: int, group: int):
    """Checks the tensors both weight formats share; returns (shape, workspace, out)."""
    _need(x, "x", torch.bfloat16)
    T, d = x.shape
    dev = x.device
    k = idx.shape[-1]
    _need(idx, "idx", torch.int32, (T, k), dev)
    _need(gates, "gates", torch.float32, (T, k), dev)
    sh = MoEShape(T, d, F, E, k)
    nbytes = load().dg_moe_swiglu_workspace_bytes(ctypes.byref(sh), group)
    if workspace is None:
        workspace = _scratch(dev, nbytes)
    elif nbytes:
        _need_workspace(workspace, nbytes, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", torch.bfloat16, (T, d), dev)
    return sh, workspace, out


def moe_swiglu(x: torch.Tensor, idx: torch.Tensor, gates: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j gates[t, j] * w2[e] (silu(w1[e] x[t]) * (w3[e] x[t])), e = idx[t, j], for few tokens.

    x [T, d], w13 [E, 2F, d] (rows [w1; w3]), w2 [E, d, F] bf16; idx [T, k]
    int32 and gates [T, k] binary32 as moe_route returns them (an idx outside
    [0, E) is no expert and adds nothing).  T * k <= 8192.  `workspace`
    (dg_moe_swiglu_workspace_bytes, its error block zeroed; default: this
    stream's own) is not shared by calls that run at the same time."""
    lib = load()
    d = x.shape[-1]
    E, F = w13.shape[0], w13.shape[1] // 2
    _need(w13, "w13", torch.bfloat16, (E, 2 * F, d), x.device)
    _need(w2, "w2", torch.bfloat16, (E, d, F), x.device)
    sh, workspace, out = _moe_args(x, idx, gates, workspace, out, F, E, 0)
    _launch(lib.dg_moe_swiglu, x.device, ctypes.byref(sh), _p(x), _p(idx), _p(gates), _p(w13), _p(w2), _p(out),
            _p(workspace), workspace.numel())
    return out


def moe_swiglu_w4(x: torch.Tensor, idx: torch.Tensor, gates: torch.Tensor, w13, w2,
                  workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_swiglu with 4-bit experts: w13 and w2 are (codes, scales, zeros) of [E, 2F, d] and [E, d, F]
    (w4_quantize of the bf16 tensors), of one group size, both with zero points or both without."""
    lib = load()
    d, dev = x.shape[-1], x.device
    (c13, s13, z13), (c2, s2, z2) = w13, w2
    E, F = c13.shape[0], c13.shape[1] // 2
    group = _need_w4(c13, s13, z13, (E, 2 * F), d, dev, "w13 ")
    if _need_w4(c2, s2, z2, (E, d), F, dev, "w2 ") != group:
        raise ValueError("w13 and w2 must have the same group size")
    sh, workspace, out = _moe_args(x, idx, gates, workspace, out, F, E, group)
    _launch(lib.dg_moe_swiglu_w4, dev, ctypes.byref(sh), group, _p(x), _p(idx), _p(gates), _p(c13), _p(s13), _p(z13),
            _p(c2), _p(s2), _p(z2), _p(out), _p(workspace), workspace.numel())
    return out


def moe_layer(x: torch.Tensor, w_router: torch.Tensor, w13, w2, top_k: int, score: str = "softmax",
              renormalize: bool = True, scale: float = 1.0, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A whole routed layer for few tokens: moe_route, then moe_swiglu (bf16 w13, w2) or moe_swiglu_w4
    (w13, w2 as (codes, scales, zeros))."""
    idx, gates = moe_route(x, w_router, top_k, score, renormalize, scale)
    call = moe_swiglu if isinstance(w13, torch.Tensor) else moe_swiglu_w4
    return call(x, idx, gates, w13, w2, workspace=workspace)

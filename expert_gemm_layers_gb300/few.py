"""Torch-facing wrappers of the few-token operators: 4-bit weights and routed experts.

As in ops.py, each function checks its arguments, allocates outputs and
scratch with torch and passes pointers and the current stream to the C ABI.
Weights in 4 bits are (codes, scales, zeros) as w4_quantize returns them:
codes [..., K/2] uint8, scales [..., K/group] bf16, zeros [..., K/group] uint8
or None (zero point 8).  None of these operators has a backward: inputs that
require gradients are taken as constants, and refused by moe_layer.
"""
from __future__ import annotations

import threading

import torch

from ._lib import DG_ERROR_BLOCK_BYTES, DG_MOE_RENORM, DG_MOE_SIGMOID, MoEShape, check, load
from .ops import _need, alloc_workspace

__all__ = ["w4_quantize", "w4_dequantize", "w4_linear", "moe_route", "moe_swiglu", "moe_swiglu_w4", "moe_layer"]


# A decode step makes many of these calls, each a few microseconds of GPU work,
# so what the host does per call is kept short: one expression per tensor (the
# slow, exact check runs only to say what is wrong) and the stream as a number.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing
BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


def _device(x, name: str, dtype) -> int:
    """The index of the device that the call runs on: that of its first tensor."""
    index = x.get_device() if isinstance(x, torch.Tensor) else -1
    if index < 0:
        _need(x, name, dtype)
    return index


def _check(t, name: str, dtype, shape, index: int) -> None:
    """_need(t, name, dtype, shape, device `index`), fast where nothing is wrong."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, shape, torch.device("cuda", index))


def _launch(fn, index: int, *args) -> None:
    """fn(*args, current stream) with device `index` current."""
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        check(status)


def _size(t, dim: int) -> int:
    """Size of a dimension; 0 for what has no such dimension, which the check of its shape then refuses."""
    return t.shape[dim] if isinstance(t, torch.Tensor) and -t.dim() <= dim < t.dim() else 0


def _p(t):
    return None if t is None else t.data_ptr()


_scratch_cache: dict = {}
_KEEP_BYTES = 64 << 20


def _scratch(index: int, stream: int, nbytes: int) -> torch.Tensor:
    """The workspace this module gives calls that bring none: one per (device,
    current stream), grown as needed, its error block zeroed when it is made.
    A captured call gets one of its own, in the graph's memory, so that graphs
    captured on one stream do not share it; a call that needs more than
    _KEEP_BYTES gets one that goes back to torch after it (calls of that size take
    far longer than to zero an error block).  Device `index` is current."""
    if nbytes > _KEEP_BYTES or _is_capturing():
        return alloc_workspace(nbytes, torch.device("cuda", index))
    key = (index, stream)
    ws = _scratch_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _scratch_cache[key] = alloc_workspace(nbytes, torch.device("cuda", index))
    return ws


def _need_workspace(ws: torch.Tensor, nbytes: int, index: int) -> None:
    _check(ws, "workspace", U8, ws.shape if isinstance(ws, torch.Tensor) else None, index)
    if ws.numel() < nbytes:
        raise ValueError(f"workspace has {ws.numel()} bytes, needs {nbytes}")


# Threads can have the same current stream, and a call is several kernels: those of two calls
# on this module's workspace are not to mix.
_scratch_lock = threading.RLock()


def _launch_with(workspace, nbytes: int, fn, index: int, *args) -> None:
    """_launch with a workspace of at least `nbytes` as the last arguments: the caller's, or (None) this module's."""
    if workspace is not None:
        _need_workspace(workspace, nbytes, index)
        _launch(fn, index, *args, workspace.data_ptr(), workspace.numel())
        return
    if _current_device() != index:
        with torch.cuda.device(index):
            _launch_with(None, nbytes, fn, index, *args)
        return
    stream = _raw_stream(index)
    with _scratch_lock:
        workspace = _scratch(index, stream, nbytes)
        status = fn(*args, workspace.data_ptr(), workspace.numel(), stream)
    if status:
        check(status)


# ------------------------------------------------------------------ 4-bit weights

def _need_w4(codes, scales, zeros, lead: tuple, K: int, index: int, what: str) -> int:
    """Checks one 4-bit weight [*lead, K]; returns its group size."""
    _check(codes, what + "codes", U8, (*lead, K // 2), index)
    groups = _size(scales, -1)
    if groups < 1 or K % groups:
        raise ValueError(f"{what}scales must be [..., K/group] beside codes [..., K/2]")
    _check(scales, what + "scales", BF16, (*lead, groups), index)
    if zeros is not None:
        _check(zeros, what + "zeros", U8, scales.shape, index)
    return K // groups


def w4_quantize(weight: torch.Tensor, group: int = 128, zero_points: bool = False):
    """4-bit codes of a bf16 weight [..., K] with one scale per `group` columns (32, 64 or 128).

    Returns (codes, scales, zeros): value = (code - zero) * scale.  zeros is
    None unless zero_points (then codes span each group's own range instead of
    a symmetric one)."""
    index = _device(weight, "weight", BF16)
    _check(weight, "weight", BF16, weight.shape, index)
    lead, K = weight.shape[:-1], _size(weight, -1)
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide {K}, got {group}")
    codes = torch.empty((*lead, K // 2), dtype=U8, device=weight.device)
    scales = torch.empty((*lead, K // group), dtype=BF16, device=weight.device)
    zeros = torch.empty((*lead, K // group), dtype=U8, device=weight.device) if zero_points else None
    _launch(load().dg_w4_quantize, index, weight.numel() // K if K else 0, K, group, weight.data_ptr(),
            codes.data_ptr(), scales.data_ptr(), _p(zeros))
    return codes, scales, zeros


def w4_dequantize(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 weight [..., K] that 4-bit codes stand for."""
    index = _device(codes, "codes", U8)
    lead, K = codes.shape[:-1], 2 * _size(codes, -1)
    group = _need_w4(codes, scales, zeros, lead, K, index, "")
    if out is None:
        out = torch.empty((*lead, K), dtype=BF16, device=scales.device)
    else:
        _check(out, "out", BF16, (*lead, K), index)
    _launch(load().dg_w4_dequantize, index, out.numel() // K if K else 0, K, group, codes.data_ptr(),
            scales.data_ptr(), _p(zeros), out.data_ptr())
    return out


def w4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W^T (+ bias) with W [out, in] in 4 bits, for few rows x [..., in] (a decode step).

    Sums in binary32, one rounding to bf16.  For long prompts dequantise once
    and use tp_linear.  `ws` holds the call's error block (default: this
    stream's own), and scratch where there are more than few short rows
    (dg_w4_linear_workspace_bytes)."""
    lib, index = load(), _device(x, "x", BF16)
    lead, in_f, out_f = x.shape[:-1], _size(x, -1), _size(codes, 0)
    _check(x, "x", BF16, x.shape, index)
    group = _need_w4(codes, scales, zeros, (out_f,), in_f, index, "")
    if bias is not None:
        _check(bias, "bias", BF16, (out_f,), index)
    if out is None:
        out = torch.empty((*lead, out_f), dtype=BF16, device=x.device)
    else:
        _check(out, "out", BF16, (*lead, out_f), index)
    rows = x.numel() // in_f if in_f else 0
    _launch_with(ws, lib.dg_w4_linear_workspace_bytes(rows, in_f, out_f), lib.dg_w4_linear, index, rows, in_f, out_f,
                 group, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), _p(zeros), _p(bias), out.data_ptr())
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
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    lib, index = load(), _device(x, "x", BF16)
    T, d, E = _size(x, 0), _size(x, -1), _size(w_router, 0)
    _check(x, "x", BF16, (T, d), index)
    _check(w_router, "w_router", BF16, (E, d), index)
    flags = (DG_MOE_SIGMOID if score == "sigmoid" else 0) | (DG_MOE_RENORM if renormalize else 0)
    idx = torch.empty((T, top_k), dtype=I32, device=x.device)
    gates = torch.empty((T, top_k), dtype=F32, device=x.device)
    _launch_with(workspace, lib.dg_moe_route_workspace_bytes(T, d, E, top_k), lib.dg_moe_route, index, T, d, E, top_k,
                 flags, scale, x.data_ptr(), w_router.data_ptr(), idx.data_ptr(), gates.data_ptr())
    return idx, gates


def _moe_args(index, x, idx, gates, out, F: int, E: int, group: int):
    """Checks the tensors both weight formats share; returns (shape, workspace bytes, out)."""
    T, d, k = _size(x, 0), _size(x, -1), _size(idx, -1)
    _check(x, "x", BF16, (T, d), index)
    _check(idx, "idx", I32, (T, k), index)
    _check(gates, "gates", F32, (T, k), index)
    sh = MoEShape(T, d, F, E, k)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", BF16, (T, d), index)
    return sh, load().dg_moe_swiglu_workspace_bytes(sh, group), out


def moe_swiglu(x: torch.Tensor, idx: torch.Tensor, gates: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j gates[t, j] * w2[e] (silu(w1[e] x[t]) * (w3[e] x[t])), e = idx[t, j], for few tokens.

    x [T, d], w13 [E, 2F, d] (rows [w1; w3]), w2 [E, d, F] bf16; idx [T, k]
    int32 and gates [T, k] binary32 as moe_route returns them (an idx outside
    [0, E) is no expert and adds nothing).  T * k <= 8192.  `workspace`
    (dg_moe_swiglu_workspace_bytes, its error block zeroed; default: this
    stream's own) is not shared by calls that run at the same time."""
    index, d = _device(x, "x", BF16), _size(x, -1)
    E, F = _size(w13, 0), _size(w13, 1) // 2
    _check(w13, "w13", BF16, (E, 2 * F, d), index)
    _check(w2, "w2", BF16, (E, d, F), index)
    sh, nbytes, out = _moe_args(index, x, idx, gates, out, F, E, 0)
    _launch_with(workspace, nbytes, load().dg_moe_swiglu, index, sh, x.data_ptr(), idx.data_ptr(), gates.data_ptr(),
                 w13.data_ptr(), w2.data_ptr(), out.data_ptr())
    return out


def moe_swiglu_w4(x: torch.Tensor, idx: torch.Tensor, gates: torch.Tensor, w13, w2,
                  workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_swiglu with 4-bit experts: w13 and w2 are (codes, scales, zeros) of [E, 2F, d] and [E, d, F]
    (w4_quantize of the bf16 tensors), of one group size, both with zero points or both without."""
    index, d = _device(x, "x", BF16), _size(x, -1)
    (c13, s13, z13), (c2, s2, z2) = w13, w2
    E, F = _size(c13, 0), _size(c13, 1) // 2
    group = _need_w4(c13, s13, z13, (E, 2 * F), d, index, "w13 ")
    if _need_w4(c2, s2, z2, (E, d), F, index, "w2 ") != group:
        raise ValueError("w13 and w2 must have the same group size")
    sh, nbytes, out = _moe_args(index, x, idx, gates, out, F, E, group)
    _launch_with(workspace, nbytes, load().dg_moe_swiglu_w4, index, sh, group, x.data_ptr(), idx.data_ptr(),
                 gates.data_ptr(), c13.data_ptr(), s13.data_ptr(), _p(z13), c2.data_ptr(), s2.data_ptr(), _p(z2),
                 out.data_ptr())
    return out


def moe_layer(x: torch.Tensor, w_router: torch.Tensor, w13, w2, top_k: int, score: str = "softmax",
              renormalize: bool = True, scale: float = 1.0, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A whole routed layer for few tokens: moe_route, then moe_swiglu (bf16 w13, w2) or moe_swiglu_w4
    (w13, w2 as (codes, scales, zeros)).  T * top_k <= 8192, as theirs: split a longer prompt by tokens.
    `workspace` is the experts' (the router takes this stream's own).

    Unlike the other *_layer functions it is not differentiable: tensors that require gradients are
    refused where autograd records (run it under torch.no_grad())."""
    if torch.is_grad_enabled():
        weights = [t for w in (w13, w2) for t in (w if isinstance(w, (tuple, list)) else (w,))]
        if any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, w_router, *weights)):
            raise RuntimeError("moe_layer has no backward: run it under torch.no_grad(), or detach its inputs")
    idx, gates = moe_route(x, w_router, top_k, score, renormalize, scale)
    call = moe_swiglu if isinstance(w13, torch.Tensor) else moe_swiglu_w4
    return call(x, idx, gates, w13, w2, workspace=workspace)

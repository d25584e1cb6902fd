"""Torch-facing wrappers of the block-scaled e4m3 operators: quantiser, linear, root-mean-square norm.

As in ops.py, each function checks its arguments, allocates outputs and
scratch with torch and passes pointers and the current stream to the C ABI.
A matrix in this format is a pair (codes, scales): codes float8_e4m3fn
[..., K], scales float8_e8m0fnu with one power of two for every 128 columns of
a row (activations: [..., ceil(K/128)]) or every 128 x 128 block (weights
[N, K]: [ceil(N/128), ceil(K/128)]); value = code * scale.

The *_layer functions are differentiable and keep activations in 8 bits for
the backward; in the others, inputs that require gradients are taken as
constants.  A layer's backward can be captured into a graph with
torch.autograd.grad; no gradient of a gradient.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import load
from .few import BF16, _check, _device, _launch, _launch_with, _p, _size
from .ops import tp_linear, tp_linear_backward, tp_swiglu, tp_swiglu_backward

__all__ = ["fp8_quantize", "fp8_dequantize", "fp8_linear", "fp8_linear_backward", "FP8Linear", "fp8_linear_layer",
           "rms_norm", "rms_norm_backward", "RMSNorm", "rms_norm_layer", "FP8NormLinear", "fp8_norm_linear_layer",
           "TPLinearKeep8", "tp_linear_layer_keep8", "TPSwiGLUKeep8", "tp_swiglu_layer_keep8"]

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _pair(pair, what: str):
    if not (isinstance(pair, (tuple, list)) and len(pair) == 2):
        raise TypeError(f"{what} must be (codes, scales)")
    return pair


# As in few.py: one expression where nothing is wrong, the exact checks only to say what is.

def _held(pair, what: str) -> tuple:
    """Checks activations in 8 bits; returns (codes, scales, device index, leading sizes, rows, d)."""
    codes, scales = _pair(pair, what)
    if isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and codes.dim():
        shape, index = codes.shape, codes.get_device()
        lead, d = shape[:-1], shape[-1]
        if codes.dtype is E4M3 and scales.dtype is E8M0 and 0 <= index == scales.get_device() and \
                scales.shape == (*lead, (d + 127) // 128) and codes.is_contiguous() and scales.is_contiguous():
            return codes, scales, index, lead, codes.numel() // d if d else 0, d
    index = _device(codes, f"{what} codes", E4M3)
    _check(codes, f"{what} codes", E4M3, codes.shape, index)
    _check(scales, f"{what} scales", E8M0, (*codes.shape[:-1], _blocks(_size(codes, -1))), index)
    raise ValueError(f"{what} codes must have a last dimension")


def _need_weight(pair, what: str, in_f: int, index: int) -> tuple:
    """Checks a weight [out, in_f] in 8 bits; returns (codes, scales, out)."""
    codes, scales = _pair(pair, what)
    out_f = _size(codes, 0)
    if not (out_f and isinstance(scales, torch.Tensor) and codes.dtype is E4M3 and scales.dtype is E8M0
            and codes.shape == (out_f, in_f) and scales.shape == ((out_f + 127) // 128, (in_f + 127) // 128)
            and codes.get_device() == index == scales.get_device() and codes.is_contiguous() and scales.is_contiguous()):
        _check(codes, f"{what} codes", E4M3, (out_f, in_f), index)
        _check(scales, f"{what} scales", E8M0, (_blocks(out_f), _blocks(in_f)), index)
    return codes, scales, out_f


def _rows(t) -> int:
    return t.numel() // t.shape[-1] if t.dim() and t.shape[-1] else 0


def _activations(x, name: str) -> tuple:
    """Checks a contiguous bf16 CUDA tensor [..., d]; returns (device index, leading sizes, rows, d)."""
    index = _device(x, name, BF16)
    if x.dtype is not BF16 or not x.is_contiguous() or not x.dim():
        _check(x, name, BF16, x.shape, index)
        raise ValueError(f"{name} must have a last dimension")
    shape = x.shape
    d = shape[-1]
    return index, shape[:-1], x.numel() // d if d else 0, d


# ------------------------------------------------------------------ the format

def fp8_quantize(x: torch.Tensor, block_rows: int = 1):
    """(codes, scales) of a bf16 tensor: one scale per 128 columns of a row (block_rows 1, x [..., K]) or per
    128 x 128 block (block_rows 128, x [N, K]).  K % 16 == 0.

    A scale is the least power of two (from 2^-124) for which no code exceeds 448, 1 for a block of zeros; a block
    with a NaN or an infinity becomes NaN."""
    index, lead, rows, K = _activations(x, "x")
    if block_rows != 1:
        if block_rows != 128 or x.dim() != 2:
            raise ValueError(f"block_rows must be 1, or 128 with x [N, K]; got {block_rows} with shape {tuple(x.shape)}")
        lead = (_blocks(rows),)
    codes = torch.empty(x.shape, dtype=E4M3, device=x.device)
    scales = torch.empty((*lead, _blocks(K)), dtype=E8M0, device=x.device)
    _launch(load().dg_fp8_quantize, index, rows, K, block_rows, x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def fp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 tensor that (codes, scales) stand for.  scales [..., ceil(K/128)] is read as activations' and
    [ceil(N/128), ceil(K/128)] beside codes [N, K] as a weight's (one row is both)."""
    index = _device(codes, "codes", E4M3)
    _check(codes, "codes", E4M3, codes.shape, index)
    K, rows = _size(codes, -1), _rows(codes)
    as_rows = (*codes.shape[:-1], _blocks(K))
    block_rows = 1
    if codes.dim() == 2 and isinstance(scales, torch.Tensor) and scales.shape != as_rows:
        as_rows, block_rows = (_blocks(rows), _blocks(K)), 128
    _check(scales, "scales", E8M0, as_rows, index)
    if out is None:
        out = torch.empty(codes.shape, dtype=BF16, device=codes.device)
    else:
        _check(out, "out", BF16, codes.shape, index)
    _launch(load().dg_fp8_dequantize, index, rows, K, block_rows, codes.data_ptr(), scales.data_ptr(), out.data_ptr())
    return out


# ------------------------------------------------------------------ linear

def fp8_linear(x, weight, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = x @ W^T (+ bias) in block-scaled e4m3, from one row (a decode step) to whole prompts.

    x: activations in 8 bits (codes, scales), as fp8_quantize and rms_norm(..., fp8=True) return them, or bf16
    [..., in], which is quantised on the way.  weight: (codes, scales) of fp8_quantize(W [out, in], 128).  Sums in
    binary32, one rounding to bf16.  Inputs that require gradients are taken as constants (fp8_linear_layer is the
    differentiable form).  `workspace` (dg_fp8_linear_workspace_bytes, or for bf16 dg_fp8_linear_bf16_workspace_bytes;
    its error block zeroed; default: this stream's own) is not shared by calls that run at the same time."""
    lib = load()
    if isinstance(x, torch.Tensor):
        index, lead, rows, in_f = _activations(x, "x")
        xc, xs = x, None
    else:
        xc, xs, index, lead, rows, in_f = _held(x, "x")
    wc, wscale, out_f = _need_weight(weight, "weight", in_f, index)
    if bias is not None:
        _check(bias, "bias", BF16, (out_f,), index)
    if out is None:
        out = torch.empty((*lead, out_f), dtype=BF16, device=xc.device)
    else:
        _check(out, "out", BF16, (*lead, out_f), index)
    if xs is None:
        _launch_with(workspace, lib.dg_fp8_linear_bf16_workspace_bytes(rows, in_f, out_f), lib.dg_fp8_linear_bf16, index,
                     rows, in_f, out_f, x.data_ptr(), wc.data_ptr(), wscale.data_ptr(), _p(bias), out.data_ptr())
    else:
        _launch_with(workspace, lib.dg_fp8_linear_workspace_bytes(rows, in_f, out_f), lib.dg_fp8_linear, index, rows,
                     in_f, out_f, xc.data_ptr(), xs.data_ptr(), wc.data_ptr(), wscale.data_ptr(), _p(bias),
                     out.data_ptr())
    return out


def fp8_linear_backward(x, weight, dy: torch.Tensor, need_dx: bool = True, need_dw: bool = True,
                        need_db: bool = False, workspace: torch.Tensor | None = None) -> dict:
    """Gradients of fp8_linear from the 8-bit operands that the forward read, given dy [..., out] bf16.

    "x" = q(dy) W, where q(dy) is dy through fp8_quantize, "weight" = dy^T x (dy as it is), "bias" = column sums of
    dy; bf16, None where not needed.  x and weight may be None where their products are not needed.  `workspace`
    (dg_fp8_linear_bwd_workspace_bytes_for) as in fp8_linear; scratch is that of the gradients asked for."""
    lib, (index, lead, rows, out_f) = load(), _activations(dy, "dy")
    xc = xs = wc = ws = None
    if x is None and need_dw or weight is None and need_dx:
        raise ValueError("x is needed for the weight's gradient, weight for that of x")
    in_f = 16  # where neither is given, for the bias's gradient: it has no part in that
    if x is not None:
        xc, xs, at, *_ = _held(x, "x")
        if xc.shape[:-1] != lead or at != index:
            raise ValueError(f"x codes have shape {tuple(xc.shape)} on device {at} beside dy {tuple(dy.shape)} on {index}")
        in_f = xc.shape[-1]
    if weight is not None:
        in_f = in_f if x is not None else _size(_pair(weight, "weight")[0], -1)
        wc, ws, n = _need_weight(weight, "weight", in_f, index)
        if n != out_f:
            raise ValueError(f"weight codes have shape {tuple(wc.shape)} beside dy {tuple(dy.shape)}")
    new = lambda shape: torch.empty(shape, dtype=BF16, device=dy.device)
    g = dict(x=new((*lead, in_f)) if need_dx else None, weight=new((out_f, in_f)) if need_dw else None,
             bias=new((out_f,)) if need_db else None)
    need = lib.dg_fp8_linear_bwd_workspace_bytes_for(rows, in_f, out_f, bool(need_dx), bool(need_dw), bool(need_db))
    _launch_with(workspace, need, lib.dg_fp8_linear_bwd, index, rows, in_f, out_f, _p(xc), _p(xs), _p(wc), _p(ws),
                 dy.data_ptr(), _p(g["x"]), _p(g["weight"]), _p(g["bias"]))
    return g


def _pair_or_none(codes, scales):
    return None if codes is None else (codes, scales)


_NO_PAIR = (None, None)


class FP8Linear(torch.autograd.Function):
    """Autograd wrapper of fp8_linear on bf16 tensors: quantises both operands and keeps, in 8 bits, those that the
    gradients asked for read."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        x8, w8 = fp8_quantize(x), fp8_quantize(weight, 128)
        need_x, need_w, _ = ctx.needs_input_grad
        ctx.save_for_backward(*(x8 if need_w else _NO_PAIR), *(w8 if need_x else _NO_PAIR))
        return fp8_linear(x8, w8, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        xc, xs, wc, ws = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = fp8_linear_backward(_pair_or_none(xc, xs), _pair_or_none(wc, ws), dy.contiguous(), *need)
        return g["x"], g["weight"], g["bias"]


def fp8_linear_layer(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable y = x @ weight^T (+ bias): x [..., in], weight [out, in] and bias bf16, products in block-scaled
    e4m3.  Of x the backward keeps 8 bits a value, nothing where the weight is frozen; its gradients are
    fp8_linear_backward's, passed through the quantisers."""
    return FP8Linear.apply(x, weight, bias)


# ------------------------------------------------------------------ root-mean-square norm

def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
             fp8: bool = False):
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, h = x + residual (bf16).

    y is bf16, or with fp8 activations in 8 bits (codes, scales) for fp8_linear, from the binary32 values.  Inputs that
    require gradients are taken as constants (rms_norm_layer is the differentiable form).  Returns y, or (y, h) where a
    residual is given.  x, residual [..., d], weight [d] bf16; d % 8 == 0 (16 with fp8), d <= 32768, eps >= 1e-30."""
    index, lead, rows, d = _activations(x, "x")
    _check(weight, "weight", BF16, (d,), index)
    h = y = codes = scales = None
    if residual is not None:
        _check(residual, "residual", BF16, x.shape, index)
        h = torch.empty_like(x)
    if fp8:
        codes = torch.empty(x.shape, dtype=E4M3, device=x.device)
        scales = torch.empty((*lead, _blocks(d)), dtype=E8M0, device=x.device)
    else:
        y = torch.empty_like(x)
    _launch(load().dg_rms_norm, index, rows, d, eps, x.data_ptr(), _p(residual), weight.data_ptr(), _p(h), _p(y),
            _p(codes), _p(scales))
    y = (codes, scales) if fp8 else y
    return y if residual is None else (y, h)


def rms_norm_backward(h: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, dh: torch.Tensor | None = None,
                      eps: float = 1e-6, need_dx: bool = True, need_dw: bool = True,
                      workspace: torch.Tensor | None = None) -> dict:
    """Gradients of rms_norm from h (x, where there was no residual), dy and, if h had other uses, their gradient dh:
    "x" (also the residual's) and "weight", bf16."""
    lib, (index, _, rows, d) = load(), _activations(h, "h")
    _check(weight, "weight", BF16, (d,), index)
    _check(dy, "dy", BF16, h.shape, index)
    if dh is not None:
        _check(dh, "dh", BF16, h.shape, index)
    g = dict(x=torch.empty_like(h) if need_dx else None, weight=torch.empty_like(weight) if need_dw else None)
    _launch_with(workspace, lib.dg_rms_norm_bwd_workspace_bytes(rows, d), lib.dg_rms_norm_bwd, index, rows, d, eps,
                 h.data_ptr(), weight.data_ptr(), dy.data_ptr(), _p(dh), _p(g["x"]), _p(g["weight"]))
    return g


def _norm_grads(h, weight, dy, dh, eps, need):
    """(dx, d_weight, d_residual) of a norm for needs (x, weight, residual); dy or dh None: no gradient came that way."""
    dh = None if dh is None else dh.contiguous()
    if dy is None:  # h alone was used: the sum passes its gradient on
        g = dict(x=dh, weight=torch.zeros_like(weight) if need[1] else None)
    else:
        g = rms_norm_backward(h, weight, dy.contiguous(), dh, eps, need[0] or need[2], need[1])
    return g["x"] if need[0] else None, g["weight"], g["x"] if need[2] else None


class RMSNorm(torch.autograd.Function):
    """Autograd wrapper of rms_norm with a bf16 result; keeps h and the weight."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        out = rms_norm(x, weight, residual, eps)
        ctx.save_for_backward(x if residual is None else out[1], weight)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        return (*_norm_grads(*ctx.saved_tensors, dy, dh, ctx.eps, ctx.needs_input_grad), None)


def rms_norm_layer(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """Differentiable rms_norm (bf16 result): y, or (y, h) with a residual."""
    return RMSNorm.apply(x, weight, residual, eps)


class FP8NormLinear(torch.autograd.Function):
    """Norm, then linear, the normalised activations in 8 bits between them and for the backward."""

    @staticmethod
    def forward(ctx, x, norm_weight, weight, bias, residual, eps):
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        normed = rms_norm(x, norm_weight, residual, eps, fp8=True)
        n8, h = normed if residual is not None else (normed, x)
        w8 = fp8_quantize(weight, 128)
        y = fp8_linear(n8, w8, bias)
        need_x, need_nw, need_w, need_b, need_r, _ = ctx.needs_input_grad
        through = need_x or need_nw or need_r
        ctx.save_for_backward(*((h, norm_weight) if through else _NO_PAIR), *(n8 if need_w else _NO_PAIR),
                              *(w8 if through else _NO_PAIR))
        ctx.weight_shape = weight.shape
        return y if residual is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, norm_weight, nc, ns, wc, ws = ctx.saved_tensors
        need_x, need_nw, need_w, need_b, need_r, _ = ctx.needs_input_grad
        through = need_x or need_nw or need_r
        if dy is None:  # h alone was used
            new = lambda shape: torch.zeros(shape, dtype=BF16, device=dh.device)
            g = dict(x=None, weight=new(ctx.weight_shape) if need_w else None, bias=new(ctx.weight_shape[:1]) if need_b else None)
        else:
            g = fp8_linear_backward(_pair_or_none(nc, ns), _pair_or_none(wc, ws), dy.contiguous(), through, need_w, need_b)
        dx = dnw = dr = None
        if through:
            dx, dnw, dr = _norm_grads(h, norm_weight, g["x"], dh, ctx.eps, (need_x, need_nw, need_r))
        return dx, dnw, g["weight"], g["bias"], dr, None


def fp8_norm_linear_layer(x: torch.Tensor, norm_weight: torch.Tensor, weight: torch.Tensor,
                          bias: torch.Tensor | None = None, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """Differentiable rms_norm(x + residual) @ weight^T (+ bias), the norm's result in block-scaled e4m3: y, or (y, h)
    with a residual.  Between forward and backward it keeps, of h (bf16, the residual stream itself) and of 8 bits a
    value of the norm's result and of the weight, what the gradients asked for read."""
    return FP8NormLinear.apply(x, norm_weight, weight, bias, residual, eps)


# ------------------------------------------------------------------ bf16 layers that keep 8-bit activations

def _recorded(*tensors) -> bool:
    """Whether autograd records a call on these inputs.  (Within a Function, needs_input_grad does not say that: it is
    true under torch.no_grad() too.)"""
    return torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in tensors)


class TPLinearKeep8(torch.autograd.Function):
    """tp_linear, its input kept in 8 bits for the weight's gradient (keep: a backward can follow)."""

    @staticmethod
    def forward(ctx, x, weight, bias, keep=True):
        y = tp_linear(x, weight, bias)
        ctx.save_for_backward(*(fp8_quantize(x) if keep and ctx.needs_input_grad[1] else _NO_PAIR), weight)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, scales, weight = ctx.saved_tensors
        need = ctx.needs_input_grad[:3]
        x = None if codes is None else fp8_dequantize(codes, scales)  # with a frozen weight nothing reads x
        g = tp_linear_backward(x, weight, dy.contiguous(), *need)
        return g["x"], g["weight"], g["bias"], None


def tp_linear_layer_keep8(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
    """tp_linear_layer (the same products, in bf16) that keeps 8 bits a value of x between forward and backward: the
    weight's gradient is dy^T times what the codes stand for, the others are as there.  Of x nothing is kept, and
    nothing quantised, where the weight is frozen or autograd does not record.  in % 16 == 0."""
    return TPLinearKeep8.apply(x, weight, bias, _recorded(x, weight, bias))


class TPSwiGLUKeep8(torch.autograd.Function):
    """tp_swiglu, its input kept in 8 bits (keep: a backward can follow); the backward recomputes [a|b] from these."""

    @staticmethod
    def forward(ctx, x_shards, w13, w2, keep=True):
        y = tp_swiglu(x_shards, w13, w2)
        ctx.save_for_backward(*(fp8_quantize(x_shards) if keep else _NO_PAIR), w13, w2)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, scales, w13, w2 = ctx.saved_tensors
        g = tp_swiglu_backward(fp8_dequantize(codes, scales), w13, w2, dy.contiguous())
        return g["x"], g["w13"], g["w2"], None


def tp_swiglu_layer_keep8(x_shards: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor) -> torch.Tensor:
    """tp_swiglu_layer (the same products, in bf16) that keeps 8 bits a value of x between forward and backward: its
    gradients are tp_swiglu_backward's at what the codes stand for.  Where autograd does not record, nothing is
    quantised.  d % 16 == 0."""
    return TPSwiGLUKeep8.apply(x_shards, w13, w2, _recorded(x_shards, w13, w2))

"""fp64 reference of the block-scaled e4m3 operators: quantiser, linear, root-mean-square norm.

Plain numpy on binary64 arrays.  Written from the operators' definitions in
include/dg.h; shares no code with the CUDA path.  The *_bound functions say,
per element, how far a correct result may be from the exact one.
"""
from __future__ import annotations

import numpy as np

from . import e4m3_to_f64
from .few import bf16_rne

UP = 2.0**-23   # one unit of a binary32 sum, relative
BF16 = 2.0**-8  # a rounding to bf16, relative

# finite magnitudes of e4m3 in the order of their codes 0..126
_MAGNITUDES = e4m3_to_f64(np.arange(127, dtype=np.uint8))


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 values nearest to v, |v| <= 448, ties to the even code; NaN gives 0x7f."""
    a = np.abs(np.nan_to_num(v, nan=0.0))
    hi = np.clip(np.searchsorted(_MAGNITUDES, a), 1, 126)
    lo = hi - 1
    up, down = _MAGNITUDES[hi] - a, a - _MAGNITUDES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(v), code | 0x80, code)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def scale_values(scales: np.ndarray) -> np.ndarray:
    """e8m0 bytes -> binary64."""
    s = np.asarray(scales, dtype=np.uint8).astype(np.float64)
    return np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))


def _per_element(blocks: np.ndarray, rows: int, K: int, block_rows: int) -> np.ndarray:
    return np.repeat(np.repeat(blocks, block_rows, axis=0)[:rows], 128, axis=1)[:, :K]


def quantize(x: np.ndarray, block_rows: int = 1):
    """(codes, scales), both uint8, of binary64 x [rows, K]."""
    rows, K = x.shape
    scales = np.empty((-(-rows // block_rows), -(-K // 128)), dtype=np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            b = np.abs(x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * (j + 1)])
            if not np.isfinite(b).all():
                scales[i, j] = 255
                continue
            amax, e = b.max(), -124
            while amax > 448 * 2.0**e:
                e += 1
            scales[i, j] = 127 if amax == 0 else e + 127
    with np.errstate(invalid="ignore"):
        return e4m3_codes(x / _per_element(scale_values(scales), rows, K, block_rows)), scales


def values(codes: np.ndarray, scales: np.ndarray, block_rows: int = 1) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return e4m3_to_f64(codes) * _per_element(scale_values(scales), *codes.shape, block_rows)


def product_bound(a: np.ndarray, b: np.ndarray, ref: np.ndarray) -> np.ndarray:
    """a @ b summed in binary32 over n terms, each addition off by at most one unit of a partial sum, then rounded
    to bf16 (smallest step 2^-133)."""
    err = a.shape[1] * UP * (np.abs(a) @ np.abs(b))
    return err + BF16 * (np.abs(ref) + err) + 2.0**-133


def linear(x: np.ndarray, w: np.ndarray, bias: np.ndarray | None = None):
    """(y, bound) of the values x [rows, K], w [N, K]."""
    y = x @ w.T
    err = (x.shape[1] + 1) * UP * (np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias)))
    y = y if bias is None else y + bias
    return y, err + BF16 * (np.abs(y) + err) + 2.0**-133


def linear_backward(x: np.ndarray, w: np.ndarray, dy: np.ndarray) -> dict:
    """{"x", "weight", "bias"}: (gradient, bound) each."""
    q = values(*quantize(dy))
    dx, dw, db = q @ w, dy.T @ x, dy.sum(0)
    err = dy.shape[0] * UP * np.abs(dy).sum(0)
    return dict(x=(dx, product_bound(q, w, dx)), weight=(dw, product_bound(dy.T, x, dw)),
                bias=(db, err + BF16 * (np.abs(db) + err)))


def add(x: np.ndarray, residual: np.ndarray) -> np.ndarray:
    """x + residual rounded to bf16: the sum of two bf16 values is rounded to binary32 first, which changes nothing
    that the rounding to bf16 sees unless their exponents lie over 16 apart (then by far less than half a step)."""
    return bf16_rne((x + residual).astype(np.float32))


def rms_norm(h: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * weight


# Relative error of y in binary32: a thread sums at most 32 squares one after another and at most 37 partial sums
# follow (half of it, by the root), then quotient, root, reciprocal and two products.  Each addition is counted as a
# whole unit 2^-23, though it is off by half of one at most.  That covers the backward of long rows, where a thread adds
# 128 and 13 follow: 141 halves are 70.5 units, fewer than the 32 + 37 + 8 of dx's sum; by the root 35.25, and with
# quotient and eps (0.25 each), root, reciprocal and product (0.5 each) 37.25, fewer than the 40.5 here.
NORM_REL = (32 + 37) * UP / 2 + 6 * UP


def rms_norm_bound(y: np.ndarray) -> np.ndarray:
    return (NORM_REL + BF16) * np.abs(y) + 2.0**-133


def rms_norm_backward(h, weight, dy, dh, eps: float) -> dict:
    """{"x", "weight"}: (gradient, bound) each."""
    d = h.shape[1]
    s = 1 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n, u = h * s, dy * weight
    mean = np.mean(u * n, axis=1, keepdims=True)
    inner = s * (u - n * mean)
    dx = inner if dh is None else inner + dh
    # u n summed like the squares, over magnitudes; each product and sum of the closing line once
    off = (32 + 37 + 8) * UP * np.mean(np.abs(u * n), axis=1, keepdims=True)
    err = s * (np.abs(n) * (off + 2 * NORM_REL * np.abs(mean)) + (NORM_REL + 4 * UP) * (np.abs(u) + np.abs(n * mean)))
    err = err + UP * np.abs(dx)
    dw = (dy * n).sum(0)
    errw = (h.shape[0] + 16) * UP * np.abs(dy * n).sum(0) + NORM_REL * np.abs(dy * n).sum(0)
    return dict(x=(dx, err + BF16 * (np.abs(dx) + err) + 2.0**-133),
                weight=(dw, errw + BF16 * (np.abs(dw) + errw) + 2.0**-133))

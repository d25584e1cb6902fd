"""fp64 reference of the few-token operators: 4-bit weights and routed experts.

Plain numpy on binary64 arrays (decode bf16 bit patterns with bf16_to_f64
first).  Written from the operators' definitions in include/dg.h; shares no
code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def bf16_rne(v: np.ndarray) -> np.ndarray:
    """binary32 values rounded to bf16 (nearest, ties to even), as binary64; NaN stays NaN."""
    f = np.asarray(v, dtype=np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(f), np.float32(np.nan), r).astype(np.float64)


def w4_quantize(w: np.ndarray, group: int, zero_points: bool):
    """(q [rows, K], scales [rows, K/group], zeros [rows, K/group]) of binary64 weights that are bf16 values."""
    rows, K = w.shape
    v = w.reshape(rows, K // group, group)
    f32 = np.float32
    with np.errstate(all="ignore"):
        if zero_points:
            lo, hi = np.minimum(v.min(-1), 0.0), np.maximum(v.max(-1), 0.0)
            s = bf16_rne((hi.astype(f32) - lo.astype(f32)) / f32(15))
        else:
            s = bf16_rne(np.abs(v).max(-1).astype(f32) / f32(7))
        s = np.where(s == 0, 1.0, s)
        bad = ~np.isfinite(v).all(-1) | ~np.isfinite(s)
        s = np.where(bad, np.nan, s)
        z = np.full(s.shape, 8.0)
        if zero_points:
            z = np.where(bad, 8.0, np.clip(np.rint((-lo.astype(f32)) / s.astype(f32)), 0, 15))
        q = np.rint(v.astype(f32) / s.astype(f32)[..., None]).astype(np.float64) + z[..., None]
        q = np.where(bad[..., None], z[..., None], np.clip(q, 0, 15))
    return q.reshape(rows, K).astype(np.uint8), s, z.astype(np.uint8)


def w4_pack(q: np.ndarray) -> np.ndarray:
    """Codes two to a byte, the even column in the low nibble."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def w4_unpack(codes: np.ndarray) -> np.ndarray:
    q = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=np.uint8)
    q[..., 0::2] = codes & 15
    q[..., 1::2] = codes >> 4
    return q


def w4_values(codes: np.ndarray, scales: np.ndarray, zeros: np.ndarray | None) -> np.ndarray:
    """The exact values (code - zero) * scale, binary64."""
    q = w4_unpack(codes).astype(np.float64)
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=-1)
    return (q - z) * np.repeat(scales, group, axis=-1)


def w4_magnitudes(codes: np.ndarray, scales: np.ndarray, zeros: np.ndarray | None) -> np.ndarray:
    """(code + zero) * scale: what a weight adds to the rounding error of a sum that is made as
    scale * (sum code x - zero * sum x)."""
    q = w4_unpack(codes).astype(np.float64)
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=-1)
    return (q + z) * np.repeat(np.abs(scales), group, axis=-1)


def w4_linear(x: np.ndarray, w: np.ndarray, bias: np.ndarray | None = None) -> np.ndarray:
    y = x @ w.T
    return y if bias is None else y + bias


def moe_logits(x: np.ndarray, w_router: np.ndarray) -> np.ndarray:
    """Router logits: binary64 sums rounded once to binary32 (held in binary64)."""
    return (x @ w_router.T).astype(np.float32).astype(np.float64)


def moe_choose(logits: np.ndarray, k: int, score: str = "softmax", renormalize: bool = True, scale: float = 1.0):
    """(idx [T, k], gates [T, k]) from binary32-valued logits."""
    T, E = logits.shape
    idx = np.empty((T, k), dtype=np.int32)
    gates = np.empty((T, k))
    for t in range(T):
        l = logits[t]
        # larger first, NaN behind every number, the lower index among equals
        order = sorted(range(E), key=lambda e: (np.isnan(l[e]), -l[e] if not np.isnan(l[e]) else 0.0, e))
        pick = order[:k]
        idx[t] = pick
        with np.errstate(all="ignore"):
            if np.isnan(l).any():
                gates[t] = np.nan
                continue
            if score == "sigmoid":
                log_p = -np.logaddexp(0.0, -l)    # renormalised: only in proportion, so that not all vanish
                p = np.exp(log_p - (log_p.max() if renormalize else 0.0))
            else:
                p = np.exp(l - l.max())
            if renormalize:
                total = p[pick].sum()
            else:
                total = 1.0 if score == "sigmoid" else p.sum()
            gates[t] = p[pick] / total * scale
    return idx, gates


def silu(a: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def moe_swiglu(x: np.ndarray, idx: np.ndarray, gates: np.ndarray, w13: np.ndarray, w2: np.ndarray) -> np.ndarray:
    """Routed SwiGLU experts, pair by pair; w13 [E, 2F, d], w2 [E, d, F]."""
    T, k = idx.shape
    E, F = w13.shape[0], w13.shape[1] // 2
    y = np.zeros((T, w2.shape[1]))
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if 0 <= e < E:
                a, b = w13[e, :F] @ x[t], w13[e, F:] @ x[t]
                y[t] += gates[t, j] * (w2[e] @ (silu(a) * b))
    return y


def moe_swiglu_bound(x, idx, gates, w13, w2, m13=None, m2=None) -> np.ndarray:
    """Per element, how far a correct bf16 result may be from moe_swiglu:

    * a product summed in binary32 over n terms, each addition off by at most
      one unit 2^-23 of a partial sum: n * 2^-23 * sum |w| |x|.  m13 and m2 stand
      for |w| where the sum is made of larger terms (4 bits: w4_magnitudes)
    * silu: |silu'| <= 1.1, and 2^-20 relative for exp, divide and product
    * h and y are rounded to bf16 once each: 2^-8 relative
    """
    T, k = idx.shape
    E, F = w13.shape[0], w13.shape[1] // 2
    d = x.shape[1]
    ref = moe_swiglu(x, idx, gates, w13, w2)
    err = np.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if not 0 <= e < E:
                continue
            w1, w3 = w13[e, :F], w13[e, F:]
            a, b = w1 @ x[t], w3 @ x[t]
            ax = np.abs(x[t])
            m = np.abs(w13[e]) if m13 is None else m13[e]
            da, db = d * 2.0**-23 * (m[:F] @ ax), d * 2.0**-23 * (m[F:] @ ax)
            h = silu(a) * b
            dh = 1.1 * da * (np.abs(b) + db) + np.abs(silu(a)) * db + 2.0**-20 * np.abs(h)
            dh = dh + 2.0**-8 * (np.abs(h) + dh)
            aw2, g = np.abs(w2[e]), abs(gates[t, j])
            err[t] += g * (aw2 @ dh + (F + 4) * 2.0**-23 * ((aw2 if m2 is None else m2[e]) @ (np.abs(h) + dh)))
            err[t] += (k + 2) * 2.0**-23 * g * (aw2 @ np.abs(h))
    return err + 2.0**-8 * (np.abs(ref) + err)


def moe_swiglu_by_expert(x, idx, gates, w13, w2, m13=None, m2=None):
    """(moe_swiglu, moe_swiglu_bound) of many tokens, an expert's pairs at a time.

    w13[e], w2[e], m13[e], m2[e] are the matrices of expert e: arrays, or anything indexed
    like one, so that experts can be decoded one by one."""
    T, k = idx.shape
    E = len(w13)
    ref, err = np.zeros((T, x.shape[1])), np.zeros((T, x.shape[1]))
    d, up = x.shape[1], 2.0**-23
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if t.size == 0:
            continue
        w, v = w13[e], w2[e]
        F = w.shape[0] // 2
        ax, g = np.abs(x[t]), gates[t, j][:, None]
        a, b = np.split(x[t] @ w.T, 2, axis=1)
        da, db = np.split(d * up * (ax @ (np.abs(w) if m13 is None else m13[e]).T), 2, axis=1)
        h = silu(a) * b
        dh = 1.1 * da * (np.abs(b) + db) + np.abs(silu(a)) * db + 2.0**-20 * np.abs(h)
        dh = dh + 2.0**-8 * (np.abs(h) + dh)
        av = np.abs(v)
        terms = (np.abs(h) + dh) @ (av if m2 is None else m2[e]).T
        off = np.abs(g) * (dh @ av.T + (F + 4) * up * terms + (k + 2) * up * (np.abs(h) @ av.T))
        np.add.at(ref, t, g * (h @ v.T))
        np.add.at(err, t, off)
    return ref, err + 2.0**-8 * (np.abs(ref) + err)

"""Cases of the block-scaled 8-bit operators: quantiser, linear, norm, and training on 8-bit activations.

Each case is one call (or one forward and backward) that a serving or training
loop makes.  `run` computes it in a plain form (elementary torch operations),
or, with `own` set, through the package's entry points; `exact` computes it in
64 bits.

The format: codes e4m3, value = code * scale, scale a power of two (e8m0) for
every 128 columns of a row (activations) or every 128 x 128 block (weights):
2^e with the least e >= -124 for which no code exceeds 448, 1 for a block of
zeros.  Blocks at the end of a row or column are short.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of one decoded token's block: latency
        dict(name="norm_decode", op="norm", rows=1, d=4096, res=True, fp8=False),
        # a prompt's norm with the residual's addition, written as the next product reads it (and read back)
        dict(name="norm_fp8_prompt", op="norm", rows=8192, d=4096, res=True, fp8=True),
        # norm of a training step, forward and backward, sizes off every tile
        dict(name="norm_train_odd", op="norm_train", rows=5003, d=1288, res=True),
        # a layer's w1 and w3 quantised after an optimiser step, and read back
        dict(name="quantize_ffn", op="quant", rows=28672, K=4096, block=128),
        # the fused QKV projection of one token
        dict(name="linear_decode", op="linear", rows=1, K=4096, N=6144, bias=False, pre=False),
        # the FFN's down projection of a decode batch
        dict(name="linear_few_24", op="linear", rows=24, K=14336, N=4096, bias=False, pre=False),
        # sizes off every tile, with a bias
        dict(name="linear_odd_333", op="linear", rows=333, K=1296, N=2064, bias=True, pre=False),
        # the down projection of a prompt whose activations are in 8 bits already
        dict(name="linear_prompt", op="linear", rows=8192, K=14336, N=4096, bias=False, pre=True),
        # norm and the FFN's w1 and w3 for four sequences
        dict(name="norm_linear_4", op="norm_linear", rows=4, K=4096, N=28672, res=True),
        # norm and QKV projection of a prompt
        dict(name="norm_linear_prompt", op="norm_linear", rows=8192, K=4096, N=6144, res=True),
        # a training step of norm and projection with a bias, sizes off every tile
        dict(name="train_norm_odd", op="train_norm", rows=1003, K=1296, N=2064, bias=True, res=True),
        # a training step of the FFN's first projection
        dict(name="train_ffn", op="train", rows=8192, K=4096, N=14336, bias=False),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "quant", "linear", "linear", "linear", "norm_linear", "train", "train_norm"])
    res = rng.random() < 0.75
    if op == "norm":
        fp8 = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, 8192), d=_log_int(rng, 256, 8192, 16 if fp8 else 8), res=res, fp8=fp8)
    if op == "norm_train":
        return dict(op=op, rows=_log_int(rng, 16, 8192), d=_log_int(rng, 256, 8192, 8), res=res)
    if op == "quant":
        return dict(op=op, rows=_log_int(rng, 16, 16384), K=_log_int(rng, 256, 8192, 16), block=rng.choice([1, 128]))
    train = op.startswith("train")
    while True:
        c = dict(op=op, rows=_log_int(rng, 16 if train else 1, 8192), K=_log_int(rng, 256, 8192 if "norm" in op else 14336, 16),
                 N=_log_int(rng, 256, 14336, 16))
        if c["rows"] * c["K"] * c["N"] <= 8192 * 4096 * 14336:
            break
    if op == "linear":
        c.update(bias=rng.random() < 0.5, pre=rng.random() < 0.5)
    if train:
        c.update(bias=rng.random() < 0.5)
    if "norm" in op:
        c.update(res=res)
    return c


# ------------------------------------------------------------------ inputs

def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(BF16)


def _tokens(rows, d, g):
    """Activations as a residual stream has them: a few columns are much larger than the others."""
    x = torch.randn((rows, d), generator=g, device=DEV)
    wide = torch.rand((d,), generator=g, device=DEV)
    return x.mul_(torch.where(wide > 0.995, 20.0, 1.0)).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, st = case["op"], dict(case)
    rows = case["rows"]
    if op == "quant":
        st["x"] = _randn((rows, case["K"]), g, 1.0 / math.sqrt(case["K"]))
        return st
    K = case["K"] if "K" in case else case["d"]
    st["x"] = _tokens(rows, K, g)
    if "norm" in op:
        st["r"] = _randn((rows, K), g, 2.0) if case["res"] else None
        st["g"] = (1 + 0.2 * torch.randn((K,), generator=g, device=DEV)).to(BF16)
        if "train" in op:
            st["dh"] = _randn((rows, K), g, 0.01) if case["res"] else None
    if op == "norm_train":
        st["dy"] = _randn((rows, K), g, 0.01)
    if op in ("linear", "norm_linear"):
        # a serving program holds its weights in 8 bits; they come from the format's own definition
        st["w8"] = _pack(*_codes(_randn((case["N"], K), g, 1.0 / math.sqrt(K)), 128))
        st["b"] = _randn((case["N"],), g) if case.get("bias") else None
        if case.get("pre"):
            st["x8"] = _pack(*_codes(st.pop("x"), 1))
    if op in ("train", "train_norm"):
        st["w"] = _randn((case["N"], K), g, 1.0 / math.sqrt(K))
        st["b"] = _randn((case["N"],), g) if case["bias"] else None
        st["dy"] = _randn((rows, case["N"]), g, 0.01)
    if "train" in op:
        for n in ("x", "r", "g", "w", "b"):
            if st.get(n) is not None:
                st[n].requires_grad_()
    return st


# ------------------------------------------------------------------ plain forms (binary32)

def _blocks(t, block):
    """[rows, K] padded with zeros to whole blocks, as [row blocks, block, column blocks, 128]."""
    t = torch.nn.functional.pad(t, (0, -t.shape[1] % 128, 0, -t.shape[0] % block))
    return t.view(t.shape[0] // block, block, -1, 128)


def _unblock(t, shape):
    return t.reshape(t.shape[0] * t.shape[1], -1)[:shape[0], :shape[1]]


def _codes(x, block):
    """(codes as binary32, scales as binary32) of x [rows, K]."""
    v = _blocks(x.float(), block)
    amax = v.abs().amax((1, 3))
    m, p = torch.frexp(amax.double() / 448)
    e = torch.where(m == 0.5, p - 1, p).clamp(min=-124)
    s = torch.where(amax == 0, 1.0, torch.exp2(e.double())).float()
    q = (v / s[:, None, :, None]).to(E4M3).float()
    return _unblock(q, x.shape), s


def _values(q, s, block):
    return _unblock(_blocks(q, block) * s[:, None, :, None], q.shape)


def _quantised(x, block):
    """The binary32 values that x stands for after quantisation."""
    return _values(*_codes(x, block), block)


def _pack(q, s):
    return q.to(E4M3).contiguous(), s.to(torch.float8_e8m0fnu).contiguous()


def _held(pair, block):
    return _values(pair[0].float(), pair[1].float(), block)


def _plain_norm(x, r, g):
    """(h, y in binary32): h = bf16(x + r)."""
    h = x if r is None else (x.float() + r.float()).to(BF16)
    hf = h.float()
    rstd = 1 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)
    return h, hf * rstd * g.float()


def _plain_norm_grad(dy, h, g, dh):
    """(dx, dg) for dy in binary32."""
    hf, gf = h.float(), g.float()
    rstd = 1 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)
    xhat = hf * rstd
    u = dy * gf
    dx = rstd * (u - xhat * (u * xhat).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh.float()).to(BF16), (dy * xhat).sum(0).to(BF16)


@torch.no_grad()
def _plain(op, st):
    if op == "quant":
        return _quantised(st["x"], st["block"]).to(BF16)
    if "norm" in op:
        h, y = _plain_norm(st["x"], st["r"], st["g"])
        total = () if st["r"] is None else (h,)
        if op == "norm":
            return (_quantised(y, 1).to(BF16) if st["fp8"] else y.to(BF16), *total)
        if op == "norm_train":
            return (y.to(BF16), *total, *_plain_norm_grad(st["dy"].float(), h, st["g"], st["dh"]))
    x8 = _held(st["x8"], 1) if "x8" in st else _quantised(y if "norm" in op else st["x"], 1)
    w8 = _held(st["w8"], 128) if "w8" in st else _quantised(st["w"], 128)
    out = x8 @ w8.t()
    out = (out if st.get("b") is None else out + st["b"].float()).to(BF16)
    if op == "linear":
        return out
    if op == "norm_linear":
        return (out, *total)
    dyf = st["dy"].float()
    dx = _quantised(st["dy"], 1) @ w8
    dw = (dyf.t() @ x8).to(BF16)
    db = () if st["b"] is None else (dyf.sum(0).to(BF16),)
    if op == "train":
        return (out, dx.to(BF16), dw, *db)
    dx, dg = _plain_norm_grad(dx.to(BF16).float(), h, st["g"], st["dh"])
    return (out, *total, dx, dg, dw, *db)


def run(state):
    if own:
        return _run_own(state["op"], state)
    return _plain(state["op"], state)


def _run_own(op, st):
    import expert_gemm_layers_gb300 as dg
    if op == "quant":
        return dg.fp8_dequantize(*dg.fp8_quantize(st["x"], st["block"]))
    if op == "linear":
        return dg.fp8_linear(st["x8"] if "x8" in st else st["x"], st["w8"], st["b"])
    if op == "norm":
        y = dg.rms_norm(st["x"], st["g"], st["r"], eps=EPS, fp8=st["fp8"])
        y, h = y if st["r"] is not None else (y, None)
        y = dg.fp8_dequantize(*y) if st["fp8"] else y
        return (y,) if h is None else (y, h)
    if op == "norm_linear":
        y = dg.rms_norm(st["x"], st["g"], st["r"], eps=EPS, fp8=True)
        if st["r"] is None:
            return (dg.fp8_linear(y, st["w8"]),)
        return dg.fp8_linear(y[0], st["w8"]), y[1]
    if op == "norm_train":
        out = dg.rms_norm_layer(st["x"], st["g"], st["r"], eps=EPS)
    elif op == "train":
        out = dg.fp8_linear_layer(st["x"], st["w"], st["b"])
    else:
        out = dg.fp8_norm_linear_layer(st["x"], st["g"], st["w"], st["b"], st["r"], eps=EPS)
    out = out if isinstance(out, tuple) else (out,)
    leaves = [st[n] for n in ("x", "g", "w", "b") if st.get(n) is not None]
    up = [st["dy"]] if len(out) == 1 else [st["dy"], st["dh"]]
    return (*(t.detach() for t in out), *torch.autograd.grad(out, leaves, up))


# ------------------------------------------------------------------ work

def work(case):
    op, M = case["op"], case["rows"]
    d = case.get("K", case.get("d"))
    held = 1 + 1 / 128  # bytes of an activation in 8 bits
    norm = M * d * (6 if case.get("res") else 2) + 2 * d  # x, r and h (or x), and the weight
    norm_back = M * d * (6 if case.get("res") else 4) + 4 * d + 2 * M * d  # dy, h, dh; dx; weight and its gradient
    if op == "quant":  # read the values, write the codes; read the codes, write the values
        return dict(bytes=M * d * (4 + 2 * (1 + 1 / (128 * case["block"]))), flops=3 * M * d)
    if op == "norm":
        return dict(bytes=norm + M * d * (2 * held + 2 if case["fp8"] else 2), flops=5 * M * d)
    if op == "norm_train":
        return dict(bytes=norm + 2 * M * d + norm_back, flops=15 * M * d)
    N = case["N"]
    w8 = N * d * (1 + 1 / 16384)
    bias = 2 * N if case.get("bias") else 0
    if op == "linear":
        return dict(bytes=M * d * (held if case["pre"] else 2) + w8 + 2 * M * N + bias, flops=2 * M * N * d)
    if op == "norm_linear":
        return dict(bytes=norm + w8 + 2 * M * N, flops=2 * M * N * d)
    # forward: x, w, y; backward: dy, the held x and w, dx, dw
    step = 2 * M * d + 2 * N * d + 2 * M * N + 2 * M * N + M * d * held + w8 + 2 * M * d + 2 * N * d + 2 * bias
    if op == "train_norm":
        step += norm + norm_back - 4 * M * d
    return dict(bytes=step, flops=6 * M * N * d)


# ------------------------------------------------------------------ 64 bits

def _to_e4m3(v):
    """The nearest e4m3 value of |v| <= 448, ties to even, by arithmetic."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _held64(x, block):
    """What 64-bit x [rows, K] stands for after quantisation."""
    rows, K = x.shape
    out = torch.empty_like(x)
    nb = -(-K // 128)
    peak = torch.stack([x[:, 128 * j:128 * (j + 1)].abs().max(1).values for j in range(nb)], 1)
    if block > 1:
        peak = torch.stack([peak[i:i + block].max(0).values for i in range(0, rows, block)]).repeat_interleave(block, 0)[:rows]
    e = torch.ceil(torch.log2(peak / 448)).clamp(min=-124)
    # log2 rounds: settle the exponent by the definition itself
    e = torch.where(peak > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((peak <= 448 * torch.exp2(e - 1)) & (e > -124), e - 1, e)
    s = torch.where(peak == 0, torch.ones_like(e), torch.exp2(e))
    for j in range(nb):
        c = slice(128 * j, 128 * (j + 1))
        out[:, c] = _to_e4m3(x[:, c] / s[:, j:j + 1]) * s[:, j:j + 1]
    return out


@torch.no_grad()
def exact(case, seed):
    op = case["op"]
    # weights in 8 bits were made from these very values, so their pairs are read as they stand
    st = {k: v.detach() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items()}
    if op == "quant":
        return _held64(st["x"].double(), case["block"])
    y, total = None, ()
    if "norm" in op:
        h = st["x"].double() if st["r"] is None else (st["x"].double() + st["r"].double()).to(BF16).double()
        total = () if st["r"] is None else (h,)
        inv = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        y = h * inv * st["g"].double()
        if op == "norm":
            return (_held64(y, 1) if case["fp8"] else y, *total)

    def norm_grad(dy):
        n = h * inv
        t = dy * st["g"].double()
        dx = inv * t - n * inv * torch.einsum("rd,rd->r", t, n).unsqueeze(1) / h.shape[1]
        return dx if st["dh"] is None else dx + st["dh"].double(), torch.einsum("rd,rd->d", dy, n)

    if op == "norm_train":
        return (y, *total, *norm_grad(st["dy"].double()))

    def pair(p, block):
        s = p[1].float().double().repeat_interleave(128, 1)
        s = s.repeat_interleave(block, 0) if block > 1 else s
        return p[0].float().double() * s[:p[0].shape[0], :p[0].shape[1]]

    x8 = pair(st["x8"], 1) if "x8" in st else _held64((st["x"].double() if y is None else y), 1)
    w8 = pair(st["w8"], 128) if "w8" in st else _held64(st["w"].double(), 128)
    out = torch.einsum("rk,nk->rn", x8, w8)
    out = out if st.get("b") is None else out + st["b"].double()
    if op == "linear":
        return out
    if op == "norm_linear":
        return (out, *total)
    dy = st["dy"].double()
    dx = torch.einsum("rn,nk->rk", _held64(dy, 1), w8)
    dw = torch.einsum("rn,rk->nk", dy, x8)
    db = () if st["b"] is None else (dy.sum(0),)
    if op == "train":
        return (out, dx, dw, *db)
    # the projection hands its input's gradient to the norm in bf16
    dx, dg = norm_grad(dx.to(BF16).double())
    return (out, *total, dx, dg, dw, *db)

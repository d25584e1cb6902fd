"""Cases of the few-token operators: 4-bit weights and routed experts.

Each case is one call that a serving loop makes.  `run` computes it in a plain
form (elementary torch operations), or, with `own` set, through the package's
entry points; `exact` computes it in 64 bits.

Layouts: codes [out, in/2] uint8 (low nibble = even column), scales
[out, in/group] bf16, zeros [out, in/group] uint8 or None (zero point 8);
w13 [E, 2F, d] (rows [w1; w3] of each expert), w2 [E, d, F]; idx [T, k] int32
(outside [0, E) = no expert), gates [T, k] binary32; activations bf16.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the router in front of one decoded token: latency
        dict(name="route_decode", op="route", T=1, d=4096, E=64, k=8, score="softmax", renorm=True, scale=1.0),
        # the router of a chunk of prompt tokens, sigmoid scores
        dict(name="route_chunk", op="route", T=384, d=4096, E=128, k=6, score="sigmoid", renorm=True, scale=2.5),
        # one decoded token through 8 of 64 experts (an expert = one of the SwiGLU benchmark's 8 shards)
        dict(name="moe_decode", op="moe", T=1, d=4096, F=1792, E=64, k=8, pad=0),
        # sizes off every tile, and a padded batch: the last 5 tokens have no expert
        dict(name="moe_odd_77", op="moe", T=77, d=1288, F=1400, E=60, k=6, pad=5),
        # a full decode batch: every expert's weights are read
        dict(name="moe_batch_128", op="moe", T=128, d=4096, F=1792, E=64, k=8, pad=0),
        # one decoded token, 4-bit experts
        dict(name="moe_w4_decode", op="moe_w4", T=1, d=4096, F=1792, E=64, k=8, pad=0, group=128, zeros=False),
        # a decode batch on many small 4-bit experts with zero points
        dict(name="moe_w4_batch_48", op="moe_w4", T=48, d=2048, F=768, E=128, k=8, pad=0, group=64, zeros=True),
        # the fused QKV projection of one token
        dict(name="w4_linear_decode", op="w4_linear", rows=1, K=4096, N=6144, group=128, zeros=False, bias=False),
        # the FFN's down projection for 8 sequences
        dict(name="w4_linear_8", op="w4_linear", rows=8, K=14336, N=4096, group=128, zeros=True, bias=False),
        # a wide projection with fine groups and a bias for 40 rows
        dict(name="w4_linear_40", op="w4_linear", rows=40, K=1280, N=15360, group=32, zeros=False, bias=True),
        # a layer's w1 and w3 quantised as they are loaded, and read back
        dict(name="w4_quantize_ffn", op="w4_quant", N=28672, K=4096, group=128, zeros=False),
        # a small projection with zero points, rows off every tile
        dict(name="w4_quantize_odd", op="w4_quant", N=1001, K=1312, group=32, zeros=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "moe_w4", "moe_w4", "w4_linear", "w4_linear", "w4_quant"])
    if op == "route":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log_int(rng, 1, 512), d=_log_int(rng, 256, 8192, 8), E=E, k=rng.randint(1, min(10, E)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    group = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    if op == "w4_quant":
        return dict(op=op, N=_log_int(rng, 8, 16384), K=_log_int(rng, 256, 4096, group), group=group, zeros=zeros)
    if op == "w4_linear":
        return dict(op=op, rows=_log_int(rng, 1, 64), K=_log_int(rng, 256, 16384, group), N=_log_int(rng, 256, 16384, 8),
                    group=group, zeros=zeros, bias=rng.random() < 0.5)
    while True:
        step = group if op == "moe_w4" else 8
        c = dict(op=op, T=_log_int(rng, 1, 128), d=_log_int(rng, 256, 4096, step), F=_log_int(rng, 256, 4096, step),
                 E=_log_int(rng, 4, 128), k=rng.randint(1, 8))
        c["k"] = min(c["k"], c["E"])
        c["pad"] = rng.choice([0, 0, c["T"] // 8])
        if op == "moe_w4":
            c.update(group=group, zeros=zeros)
        if c["E"] * c["d"] * c["F"] <= 64 * 4096 * 1792 and c["T"] * c["k"] * c["d"] * c["F"] <= 1024 * 4096 * 1792:
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _uniform(shape, bound, g):
    return torch.empty(shape, dtype=BF16, device=DEV).uniform_(-bound, bound, generator=g)


def _codes(lead, N, K, group, zeros, g):
    """4-bit weights as a quantiser leaves them: bell-shaped codes, scales of a few per cent spread."""
    q = torch.randn((*lead, N, K), generator=g, device=DEV, dtype=BF16).mul_(2.2).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    codes = q[..., 0::2] | (q[..., 1::2] << 4)
    s = (torch.rand((*lead, N, K // group), generator=g, device=DEV) * 0.5 + 0.75) / (2.2 * math.sqrt(3.0 * K))
    z = torch.randint(6, 11, (*lead, N, K // group), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return codes, s.to(BF16), z


def _routing(T, E, k, pad, g):
    """Distinct experts for every token with softmax gates; the last `pad` tokens are padding."""
    logit = torch.randn((T, E), generator=g, device=DEV)
    top = logit.topk(k, dim=1)
    idx, gates = top.indices.to(torch.int32), torch.softmax(top.values, dim=1)
    if pad:
        idx[T - pad:] = -1
    return idx.contiguous(), gates.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, st = case["op"], dict(case)
    if op == "route":
        st["x"] = torch.randn((case["T"], case["d"]), generator=g, device=DEV).to(BF16)
        st["w"] = _uniform((case["E"], case["d"]), math.sqrt(3.0 / case["d"]), g)
        return st
    if op == "w4_quant":
        st["w"] = torch.randn((case["N"], case["K"]), generator=g, device=DEV, dtype=BF16).mul_(1.0 / math.sqrt(case["K"]))
        return st
    if op == "w4_linear":
        st["x"] = torch.randn((case["rows"], case["K"]), generator=g, device=DEV).to(BF16)
        st["w"] = _codes((), case["N"], case["K"], case["group"], case["zeros"], g)
        st["b"] = _uniform((case["N"],), 1.0, g) if case["bias"] else None
        return st
    T, d, F, E, k = (case[n] for n in ("T", "d", "F", "E", "k"))
    st["x"] = torch.randn((T, d), generator=g, device=DEV).to(BF16)
    st["idx"], st["gates"] = _routing(T, E, k, case["pad"], g)
    if op == "moe":
        st["w13"] = _uniform((E, 2 * F, d), math.sqrt(3.0 / d), g)
        st["w2"] = _uniform((E, d, F), math.sqrt(3.0 / F), g)
    else:
        st["w13"] = _codes((E,), 2 * F, d, case["group"], case["zeros"], g)
        st["w2"] = _codes((E,), d, F, case["group"], case["zeros"], g)
    # a serving loop's scratch, zeroed once: error block, hidden rows and partial rows of every pair
    st["ws"] = torch.zeros(4096 + T * k * (2 * F + 16 * d), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms (binary32)

def _weights(w):
    """binary32 weights of bf16 weights or of (codes, scales, zeros)."""
    if torch.is_tensor(w):
        return w.float()
    codes, scales, zeros = w
    lead, groups = codes.shape[:-1], scales.shape[-1]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*lead, groups, -1).float()
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).reshape(*lead, -1)


def _pick(w, e):
    return w[e] if torch.is_tensor(w) else tuple(None if t is None else t[e] for t in w)


def _experts(w):
    return (w if torch.is_tensor(w) else w[0]).shape[0]


def _plain_moe(x, idx, gates, w13, w2):
    T, k = idx.shape
    E = _experts(w13)
    valid = (idx >= 0) & (idx < E)
    e = torch.where(valid, idx, torch.zeros_like(idx)).long()
    gt = torch.where(valid, gates, torch.zeros_like(gates))
    xf = x.float()
    if T * k <= E:  # few pairs: each pair's own weights
        e = e.reshape(-1)
        a, b = torch.bmm(_weights(_pick(w13, e)), xf.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1).chunk(2, dim=1)
        h = a / (1 + torch.exp(-a)) * b
        y = torch.bmm(_weights(_pick(w2, e)), h.unsqueeze(-1)).reshape(T, k, -1)
        return (y * gt.unsqueeze(-1)).sum(1).to(BF16)
    # many pairs: every expert on every token, weighted by the gate that the token gives it
    share = torch.zeros((T, E), device=x.device).scatter_add_(1, e, gt)
    a, b = torch.matmul(xf, _weights(w13).transpose(1, 2)).chunk(2, dim=2)
    h = a / (1 + torch.exp(-a)) * b * share.t().unsqueeze(-1)
    return torch.bmm(h, _weights(w2).transpose(1, 2)).sum(0).to(BF16)


def _plain_route(x, w, k, score, renorm, scale):
    # logits in 64 bits, rounded once: neighbours in rank can lie closer than a binary32 sum's error
    logit = (x.double() @ w.double().t()).float()
    top, idx = (v[:, :k] for v in torch.sort(logit, dim=1, descending=True, stable=True))
    if score == "softmax":
        m = logit.max(dim=1, keepdim=True).values
        p = torch.exp(top - m)
        total = p.sum(1, keepdim=True) if renorm else torch.exp(logit - m).sum(1, keepdim=True)
        gates = p / total
    else:
        gates = 1 / (1 + torch.exp(-top))
        gates = gates / gates.sum(1, keepdim=True) if renorm else gates
    return idx.to(torch.int32), gates * scale


def _plain_quantize(w, group, zeros):
    v = w.float().reshape(w.shape[0], -1, group)
    if zeros:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).to(BF16).float()
    else:
        s = (v.abs().amax(-1) / 7).to(BF16).float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = torch.round(-lo / s).clamp(0, 15) if zeros else torch.full_like(s, 8)
    q = (torch.round(v / s.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
    values = ((q - z.unsqueeze(-1)) * s.unsqueeze(-1)).to(BF16).reshape(w.shape)
    return values, s.to(BF16), z.to(torch.uint8) if zeros else None


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    if op == "route":
        return _plain_route(state["x"], state["w"], state["k"], state["score"], state["renorm"], state["scale"])
    if op == "w4_quant":
        values, scales, zeros = _plain_quantize(state["w"], state["group"], state["zeros"])
        return (values, scales) if zeros is None else (values, scales, zeros)
    if op == "w4_linear":
        y = state["x"].float() @ _weights(state["w"]).t()
        return (y if state["b"] is None else y + state["b"].float()).to(BF16)
    return _plain_moe(state["x"], state["idx"], state["gates"], state["w13"], state["w2"])


def _run_own(op, state):
    import expert_gemm_layers_gb300 as dg
    if op == "route":
        return dg.moe_route(state["x"], state["w"], state["k"], score=state["score"], renormalize=state["renorm"],
                            scale=state["scale"])
    if op == "w4_quant":
        codes, scales, zeros = dg.w4_quantize(state["w"], state["group"], zero_points=state["zeros"])
        values = dg.w4_dequantize(codes, scales, zeros)
        return (values, scales) if zeros is None else (values, scales, zeros)
    if op == "w4_linear":
        return dg.w4_linear(state["x"], *state["w"], bias=state["b"])
    call = dg.moe_swiglu if op == "moe" else dg.moe_swiglu_w4
    return call(state["x"], state["idx"], state["gates"], state["w13"], state["w2"], workspace=state["ws"])


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "route":
        T, d, E, k = (case[n] for n in ("T", "d", "E", "k"))
        return dict(bytes=2 * d * (T + E) + 8 * T * k, flops=2 * T * E * d)
    group, zeros = case.get("group", 0), case.get("zeros", False)
    per_weight = 0.5 + (3 if zeros else 2) / group if group else 2.0
    if op == "w4_quant":  # read the weights, write the codes; read the codes, write the values
        n = case["N"] * case["K"]
        return dict(bytes=n * (4 + 2 * per_weight), flops=3 * n)
    if op == "w4_linear":
        r, K, N = case["rows"], case["K"], case["N"]
        return dict(bytes=K * N * per_weight + 2 * r * (K + N) + (2 * N if case["bias"] else 0), flops=2 * r * K * N)
    T, d, F, E, k = (case[n] for n in ("T", "d", "F", "E", "k"))
    T -= case["pad"]
    touched = E * (1 - (1 - k / E) ** T)  # experts that some token picks, on average
    return dict(bytes=touched * 3 * d * F * per_weight + 4 * T * d + 8 * T * k, flops=6 * T * k * d * F)


# ------------------------------------------------------------------ 64 bits

def _unpack64(w):
    if torch.is_tensor(w):
        return w.double()
    codes, scales, zeros = w
    q = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes % 16).double()
    q[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    reps = q.shape[1] // scales.shape[1]
    z = torch.full_like(scales, 8).double() if zeros is None else zeros.double()
    return (q - z.repeat_interleave(reps, 1)) * scales.double().repeat_interleave(reps, 1)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "route":
        # the operator's logits are binary32 numbers; all that follows from them is in 64 bits
        l = torch.einsum("td,ed->te", st["x"].double(), st["w"].double()).float().double()
        order = torch.argsort(-l, dim=1, stable=True)[:, :case["k"]]
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
        gates = torch.gather(p, 1, order)
        if case["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        return order.to(torch.int32), gates * case["scale"]
    if op == "w4_linear":
        y = torch.einsum("rk,nk->rn", st["x"].double(), _unpack64(st["w"]))
        return y if st["b"] is None else y + st["b"].double()
    if op == "w4_quant":
        return _exact_quantize(st["w"], case["group"], case["zeros"])
    x, E = st["x"].double(), case["E"]
    y = torch.zeros_like(x)
    for e in range(E):
        t, j = torch.nonzero(st["idx"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        ab = x[t] @ _unpack64(_pick(st["w13"], e)).t()
        a, b = ab[:, :case["F"]], ab[:, case["F"]:]
        out = (a * torch.sigmoid(a) * b) @ _unpack64(_pick(st["w2"], e)).t()
        y.index_add_(0, t, out * st["gates"][t, j].double().unsqueeze(1))
    return y


def _exact_quantize(w, group, zeros):
    v = w.double().view(w.shape[0], w.shape[1] // group, group)
    # a scale is the bf16 value nearest to a binary32 quotient (of a binary32 difference)
    if zeros:
        lo = torch.minimum(v.min(-1).values, torch.zeros((), dtype=v.dtype, device=v.device))
        hi = torch.maximum(v.max(-1).values, torch.zeros((), dtype=v.dtype, device=v.device))
        s = ((hi - lo).float().double() / 15).float().to(BF16)
    else:
        s = (v.abs().max(-1).values / 7).float().to(BF16)
    s = s.masked_fill(s == 0, 1.0)
    s64 = s.double()
    z = (-lo / s64).round().clamp(0, 15) if zeros else 8 * torch.ones_like(s64)
    q = ((v / s64.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15)
    values = ((q - z.unsqueeze(-1)) * s64.unsqueeze(-1)).reshape(w.shape)
    return (values, s64, z.to(torch.uint8)) if zeros else (values, s64)

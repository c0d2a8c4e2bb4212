"""The operators of a mixture-of-experts layer over many tokens on 4-bit activations and 4-bit weights, as cases to measure.

Four operators; the products are in MXFP4 (32 values to an E8M0 scale) and NVFP4 (16 values to an E4M3 scale and a float32 global scale):

topk       the router's choice: scores of the experts, a bias for balance, groups, the best few, their weights
gemm       y = act(X W^T + bias) + residual of quantized activations X and quantized weights W
moe        the same for every expert's rows of a routed batch, with the gate of a gated unit in the epilogue
combine    the experts' rows back to their tokens: y[t] = residual[t] + sum_j weights[t, j] rows[dest_rows[t, j]]

`own` chooses between the plain form (elementary torch operations in float32, the router's comparisons in float64) and this package's calls.
"""
import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token's experts out of 128: latency
        dict(name="topk-1tok", op="topk", dtype="bf16", T=1, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1, sum2=False, masked=0.0),
        # a prefill batch on 384 experts in eight groups, with a bias for balance
        dict(name="topk-16384tok-grouped", op="topk", dtype="f32", T=16384, E=384, k=8, score="sigmoid", bias=True, groups=8, top_groups=4, sum2=True, masked=0.0),
        # an odd number of experts, many of them closed to a token
        dict(name="topk-odd", op="topk", dtype="f16", T=1001, E=129, k=5, score="softmax", bias=False, groups=1, top_groups=1, sum2=False, masked=0.97),
        # one token through a small projection: latency
        dict(name="gemm-1tok", op="gemm", fmt="mxfp4", dtype="bf16", T=1, N=2048, K=768, bias=True, act="none", gate="none", residual=False),
        # a decode batch through a square projection of a large hidden size, added to the residual stream
        dict(name="gemm-64tok-7168", op="gemm", fmt="nvfp4", dtype="bf16", T=64, N=7168, K=7168, bias=False, act="none", gate="none", residual=True),
        # odd rows and columns, a scale column count that is padded, an activation
        dict(name="gemm-odd", op="gemm", fmt="mxfp4", dtype="f16", T=1000, N=2881, K=2880, bias=True, act="gelu", gate="none", residual=False),
        # a prefill chunk: the tensor cores' rate
        dict(name="gemm-4096tok-7168", op="gemm", fmt="mxfp4", dtype="bf16", T=4096, N=7168, K=7168, bias=True, act="none", gate="none", residual=True),
        # gate and up products of a decode batch: nearly every expert has a few rows
        dict(name="moe-64tok-w13", op="moe", fmt="mxfp4", dtype="bf16", T=64, k=8, E=128, N=1536, K=2048, bias=False, act="silu", gate="first", drop=0.0, skew=0.0),
        # gate and up products of a prefill batch: about a thousand rows to an expert
        dict(name="moe-16384tok-w13", op="moe", fmt="mxfp4", dtype="bf16", T=16384, k=8, E=128, N=1536, K=2048, bias=True, act="silu", gate="second", drop=0.0, skew=0.0),
        # down products of a skewed routing, some routes not dispatched
        dict(name="moe-2000tok-w2-skewed", op="moe", fmt="nvfp4", dtype="f16", T=2000, k=6, E=128, N=2048, K=768, bias=True, act="none", gate="none", drop=0.1, skew=1.0),
        # one token's experts added up: latency
        dict(name="combine-1tok", op="combine", dtype="bf16", T=1, k=8, N=7168, f32=False, residual=True, drop=0.0),
        # a prefill batch: memory bandwidth
        dict(name="combine-16384tok", op="combine", dtype="bf16", T=16384, k=8, N=7168, f32=False, residual=True, drop=0.05),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("topk", "gemm", "moe", "combine"))
    if op == "topk":
        while True:
            groups = rng.choice((1, 1, 4, 8))
            c = dict(op=op, dtype=rng.choice(("bf16", "f16", "f32")), T=_log(rng, 1, 16384), E=groups * _log(rng, 8, 384 // groups), k=rng.randint(1, 8),
                     score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, top_groups=rng.randint(1, max(1, groups // 2)),
                     sum2=groups > 1 and rng.random() < 0.5, masked=rng.choice((0.0, 0.0, 0.3, 0.95)))
            if c["T"] * c["E"] <= 16384 * 384:
                return c
    if op == "combine":
        while True:
            c = dict(op=op, dtype=rng.choice(("bf16", "f16")), T=_log(rng, 1, 16384), k=rng.randint(1, 10), N=_log(rng, 64, 7168), f32=rng.random() < 0.3,
                     residual=rng.random() < 0.5, drop=rng.choice((0.0, 0.1)))
            if c["T"] * c["k"] * c["N"] * (2 if c["f32"] else 1) <= 16384 * 8 * 7168:
                return c
    fmt, dtype = rng.choice(("mxfp4", "nvfp4")), rng.choice(("bf16", "f16"))
    act, gate = rng.choice((("none", "none"), ("none", "none"), ("silu", "none"), ("gelu", "none"), ("silu", "first"), ("gelu", "second")))
    if op == "gemm":
        while True:
            c = dict(op=op, fmt=fmt, dtype=dtype, T=_log(rng, 1, 4096), N=_log(rng, 128, 8192, 1 if gate == "none" else 64), K=_log(rng, 512, 7168, 32),
                     bias=rng.random() < 0.5, act=act, gate=gate, residual=rng.random() < 0.5)
            if c["T"] * c["N"] * c["K"] <= 4096 * 7168 * 7168:
                return c
    while True:
        c = dict(op=op, fmt=fmt, dtype=dtype, T=_log(rng, 1, 16384), k=rng.choice((1, 2, 4, 6, 8)), E=_log(rng, 8, 128), N=_log(rng, 256, 4096, 8 if gate == "none" else 64),
                 K=_log(rng, 512, 4096, 32), bias=rng.random() < 0.5, act=act, gate=gate, drop=rng.choice((0.0, 0.1)), skew=rng.choice((0.0, 0.0, 1.0)))
        if c["E"] * c["N"] * c["K"] <= 128 * 1536 * 2048 and c["T"] * c["k"] * c["N"] * c["K"] <= 16384 * 8 * 1536 * 2048:
            return c


def work(c):
    if c["op"] == "topk":
        return {"bytes": c["T"] * c["E"] * (4 if c["dtype"] == "f32" else 2) + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["k"], "flops": 0}
    if c["op"] == "combine":
        routes = c["T"] * c["k"] * (1 - c["drop"])
        return {"bytes": routes * c["N"] * (4 if c["f32"] else 2) + (4 if c["residual"] else 2) * c["T"] * c["N"] + 8 * c["T"] * c["k"], "flops": 2 * routes * c["N"]}
    per = 0.5 + (1 / 32 if c["fmt"] == "mxfp4" else 1 / 16)   # bytes of a 4-bit value and its share of a scale
    N, K, out = c["N"], c["K"], c["N"] if c["gate"] == "none" else c["N"] // 2
    if c["op"] == "gemm":
        return {"bytes": (c["T"] + N) * K * per + (4 if c["residual"] else 2) * c["T"] * out + (2 * N if c["bias"] else 0), "flops": 2 * c["T"] * N * K}
    rows, used = _expected(c)
    return {"bytes": used * (N * K * per + (2 * N if c["bias"] else 0)) + rows * (K * per + 2 * out), "flops": 2 * rows * N * K}


def _popularity(c):
    """How often each expert is chosen, relative to the others: even, or falling with the expert's rank."""
    return [(e + 1.0) ** -c["skew"] for e in range(c["E"])]


def _expected(c):
    """(rows, experts that have any) of a routing, as a random one is expected to give."""
    p = _popularity(c)
    routes = min(c["k"], c["E"]) * (1 - c["drop"])
    share = [v / sum(p) for v in p]
    used = sum(1 - (1 - min(1.0, s * routes)) ** c["T"] for s in share)
    return c["T"] * routes, used


# ------------------------------------------------------- the plain forms
def _table(device):
    """Both values of each code byte, the even element first."""
    v = torch.tensor(_E2M1 + tuple(-a for a in _E2M1), device=device)
    i = torch.arange(256, device=device)
    return torch.stack((v[i % 16], v[i // 16]), 1)


def _untile(scales, rows, cols):
    """128x4-tiled scale bytes -> [rows, cols]."""
    mt, kt = -(-rows // 128), -(-cols // 4)
    return scales[:mt * kt * 512].view(mt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(mt * 128, kt * 4)[:rows, :cols]


def _tile(flat):
    """[..., rows, cols] scale bytes -> 128x4-tiled bytes [..., bytes], padded with zeros."""
    rows, cols = flat.shape[-2:]
    mt, kt = -(-rows // 128), -(-cols // 4)
    p = torch.zeros(*flat.shape[:-2], mt * 128, kt * 4, dtype=torch.uint8, device=flat.device)
    p[..., :rows, :cols] = flat
    t = p.view(*flat.shape[:-2], mt, 4, 32, kt, 4)
    n = t.dim()
    return t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).reshape(*flat.shape[:-2], -1)


def _quantize(x, fmt, g):
    """x [..., n] (16-bit values) -> packed codes [..., n/2] and scale bytes [..., n/32 or n/16], by the formats' rules in float32."""
    block = 32 if fmt == "mxfp4" else 16
    v = x.float().unflatten(-1, (-1, block))
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        e = ((top.view(torch.int32) + (1 << 21)) >> 23) & 255
        s = torch.where(e > 2, e - 2, 0).clamp(max=254)
        inv = ((254 - s) << 23).view(torch.float32)
        byte, live = s.to(torch.uint8), s > 0
    else:
        f8 = (g * (top / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte, live = f8.view(torch.uint8), f8.float() > 0
        inv = g / f8.float()
    a = torch.where(live, (v * inv).abs(), 0.0)
    # to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    c = torch.where(live & (v < 0), c + 8, c).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), byte.squeeze(-1)


def _values(codes, scales, fmt, g, table):
    """float32 values of codes [rows, n/2] with flat scale bytes."""
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float()
    else:
        s = scales.int()
        s = torch.where(s == 0, 1 << 22, s << 23).view(torch.float32)
    v = table[codes.int()].flatten(-2).unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)
    return (v if fmt == "mxfp4" else v * (1.0 / g)).flatten(-2)


def _activated(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _finished(z, c, bias, residual):
    """The epilogue: bias, activation, gate, residual."""
    if bias is not None:
        z = z + bias.to(z.dtype)
    if c["gate"] == "none":
        y = _activated(z, c["act"])
    else:
        first, second = z.chunk(2, -1)
        y = _activated(first, c["act"]) * second if c["gate"] == "first" else _activated(second, c["act"]) * first
    return y if residual is None else y + residual.to(z.dtype)


def _plain_topk(s):
    c = s["case"]
    l = s["logits"].double()
    open_ = torch.isfinite(l)
    l = torch.where(open_, l, -math.inf)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(-1, keepdim=True)
        e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
        z = e.sum(-1, keepdim=True)
        score = e / torch.where(z > 0, z, 1.0)
    pick = l
    if s["bias"] is not None:
        pick = score + s["bias"].double()
    elif c["sum2"]:
        pick = score
    pick = torch.where(open_, pick, -math.inf)
    if c["groups"] > 1:
        g = pick.view(c["T"], c["groups"], -1)
        best = g.sort(dim=-1, descending=True).values
        value = best[..., 0]
        if c["sum2"]:
            value = value + torch.where(best[..., 1] > -math.inf, best[..., 1], 0.0)
        first = value.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, first, True)
        pick = torch.where(kept.unsqueeze(-1), g, -math.inf).flatten(1)
    value, at = pick.sort(dim=-1, descending=True, stable=True)
    value, at = value[:, :c["k"]], at[:, :c["k"]]
    live = value > -math.inf
    w = torch.where(live, score.gather(1, at), 0.0)
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0) * s["scale"]
    return {"ids": torch.where(live, at, -1).to(torch.int32), "weights": w.float()}


def _plain_gemm(s):
    c = s["case"]
    x = _values(s["x_codes"], _untile(s["x_scales"], c["T"], s["cols"]), c["fmt"], s["x_g"], s["e2m1"])
    w = _values(s["codes"], _untile(s["scales"], c["N"], s["cols"]), c["fmt"], s["g"], s["e2m1"])
    return _finished(x @ w.T, c, s["bias"], s["residual"]).to(s["y"].dtype)


def _plain_moe(s):
    c = s["case"]
    flat = _untile(s["x_scales"], s["padded"][-1], s["cols"])
    per = s["scales"].numel() // c["E"]
    y = s["y"]
    for e in range(c["E"]):
        lo, hi, at = s["at"][e], s["at"][e + 1], s["padded"][e]
        if lo < hi:
            gx, g = (None, None) if c["fmt"] == "mxfp4" else (s["x_g"][e], s["g"][e])
            x = _values(s["x_codes"][lo:hi], flat[at:at + hi - lo], c["fmt"], gx, s["e2m1"])
            w = _values(s["codes"][e], _untile(s["scales"][e * per:(e + 1) * per], c["N"], s["cols"]), c["fmt"], g, s["e2m1"])
            y[lo:hi] = _finished(x @ w.T, c, None if s["bias"] is None else s["bias"][e], None).to(y.dtype)
    return y


def _plain_combine(s):
    dest = s["dest"].long()
    y = torch.zeros(s["y"].shape, device=dest.device) if s["residual"] is None else s["residual"].float()
    for j in range(dest.shape[1]):
        w = torch.where(dest[:, j] >= 0, s["weights"][:, j], 0.0)
        y = y + w.unsqueeze(1) * s["rows"][dest[:, j].clamp(min=0)].float()
    return y.to(s["y"].dtype)


# --------------------------------------------------------------- inputs
def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _quantized(gen, fmt, std, rows, K, device, experts=None):
    """Normal values quantized as a checkpoint's are: codes, tiled scales and global scales, drawn in pieces."""
    g = None
    if fmt == "nvfp4":
        g = torch.full((experts or 1,), 448.0 * 6.0 / (6.0 * std), device=device)
        if experts:
            g = g * (1.0 + torch.rand(experts, device=device, generator=gen))
    codes, flat = [], []
    total = rows * (experts or 1)
    step = rows if experts else 16384
    for i, r in enumerate(range(0, total, step)):
        q, f = _quantize((torch.randn(min(step, total - r), K, device=device, generator=gen) * std).bfloat16(), fmt, None if g is None else g[i if experts else 0])
        codes.append(q)
        flat.append(f)
    codes, flat = torch.cat(codes), torch.cat(flat)
    if experts:
        codes, flat = codes.view(experts, rows, K // 2), flat.view(experts, rows, -1)
    return codes, _tile(flat).reshape(-1), g


def _prepare_topk(c, seed, device):
    gen = _generator(seed, device)
    logits = torch.randn(c["T"], c["E"], device=device, generator=gen) * 1.5
    if c["masked"]:
        logits = torch.where(torch.rand(c["T"], c["E"], device=device, generator=gen) < c["masked"], -math.inf, logits)
    bias = torch.randn(c["E"], device=device, generator=gen) * 0.05 if c["bias"] else None
    return dict(logits=logits.to(_TYPES[c["dtype"]]), bias=bias, scale=2.5, ids=torch.empty(c["T"], c["k"], dtype=torch.int32, device=device),
                weights=torch.empty(c["T"], c["k"], device=device))


def _half(gen, c, *shape, std=0.1):
    return (torch.randn(shape, device="cuda", generator=gen) * std).to(_TYPES[c["dtype"]])


def _prepare_gemm(c, seed, device):
    gen = _generator(seed, device)
    T, N, K = c["T"], c["N"], c["K"]
    out = N if c["gate"] == "none" else N // 2
    x_codes, x_scales, x_g = _quantized(gen, c["fmt"], 1.0, T, K, device)
    codes, scales, g = _quantized(gen, c["fmt"], K ** -0.5, N, K, device)
    return dict(x_codes=x_codes, x_scales=x_scales, x_g=x_g, codes=codes, scales=scales, g=g, cols=K // (32 if c["fmt"] == "mxfp4" else 16),
                bias=_half(gen, c, N) if c["bias"] else None, residual=_half(gen, c, T, out, std=1.0) if c["residual"] else None,
                y=torch.empty(T, out, device=device, dtype=_TYPES[c["dtype"]]))


def _prepare_moe(c, seed, device):
    gen = _generator(seed, device)
    T, k, E, N, K, fmt = c["T"], min(c["k"], c["E"]), c["E"], c["N"], c["K"], c["fmt"]
    out = N if c["gate"] == "none" else N // 2
    # the routing: the k largest of popularity x exponential noise, sorted by expert
    p = torch.tensor(_popularity(c), device=device)
    ids = (p / -torch.log(torch.rand(T, E, device=device, generator=gen).clamp(min=1e-20))).topk(k, 1).indices
    ids[torch.rand(T, k, device=device, generator=gen) < c["drop"]] = E
    ids = ids.reshape(-1).sort(stable=True).values
    offsets = torch.searchsorted(ids, torch.arange(E + 1, device=device)).to(torch.int32)
    at = offsets.tolist()
    padded = [0]
    for e in range(E):
        padded.append(padded[-1] + -(-(at[e + 1] - at[e]) // 128) * 128)
    # every expert's rows quantized, their scales tiled and padded to 128 rows on their own
    rows, block = T * k, 32 if fmt == "mxfp4" else 16
    x_g = None if fmt == "mxfp4" else (448.0 * 6.0 / 6.0) * (1.0 + torch.rand(E, device=device, generator=gen))
    x_codes = torch.zeros(rows, K // 2, dtype=torch.uint8, device=device)
    flat = torch.zeros(padded[-1], K // block, dtype=torch.uint8, device=device)
    where = torch.arange(at[E], device=device)
    where = where + (torch.tensor(padded, device=device) - offsets)[ids[:at[E]]]
    for r in range(0, at[E], 16384):
        m = min(16384, at[E] - r)
        x = torch.randn(m, K, device=device, generator=gen).to(_TYPES[c["dtype"]])
        x_codes[r:r + m], f = _quantize(x, fmt, None if x_g is None else x_g[ids[r:r + m]].view(-1, 1, 1))
        flat[where[r:r + m]] = f
    # the quantizers' scale buffer has room for the worst padding of any routing
    x_scales = torch.zeros((rows + 127 * E) // 128 * 128 * (-(-K // (4 * block)) * 4), dtype=torch.uint8, device=device)
    tiled = _tile(flat)
    x_scales[:tiled.numel()] = tiled
    codes, scales, g = _quantized(gen, fmt, K ** -0.5, N, K, device, experts=E)
    return dict(x_codes=x_codes, x_scales=x_scales, x_g=x_g, offsets=offsets, at=at, padded=padded, codes=codes, scales=scales, g=g, cols=K // block,
                bias=_half(gen, c, E, N) if c["bias"] else None, y=torch.zeros(rows, out, device=device, dtype=_TYPES[c["dtype"]]),
                status=torch.zeros(1, dtype=torch.int32, device=device))


def _prepare_combine(c, seed, device):
    gen = _generator(seed, device)
    T, k, N = c["T"], c["k"], c["N"]
    rows = torch.empty(T * k, N, device=device, dtype=torch.float32 if c["f32"] else _TYPES[c["dtype"]])
    for r in range(0, T * k, 16384):
        rows[r:r + 16384] = torch.randn(min(16384, T * k - r), N, device=device, generator=gen)
    dest = torch.randperm(T * k, device=device, generator=gen).view(T, k).to(torch.int32)
    dest[torch.rand(T, k, device=device, generator=gen) < c["drop"]] = -1
    weights = torch.softmax(torch.randn(T, k, device=device, generator=gen), -1)
    return dict(rows=rows, dest=dest, weights=weights, residual=_half(gen, c, T, N, std=1.0) if c["residual"] else None,
                y=torch.empty(T, N, device=device, dtype=_TYPES[c["dtype"]]), status=torch.zeros(1, dtype=torch.int32, device=device))


def prepare(case, seed):
    make = {"topk": _prepare_topk, "gemm": _prepare_gemm, "moe": _prepare_moe, "combine": _prepare_combine}[case["op"]]
    device = torch.device("cuda")
    return dict(make(case, seed, device), e2m1=_table(device), case=case)


# ----------------------------------------------------------- one pass
def _own(s):
    import mxfp4_block_quantization_gb300 as mx

    c = s["case"]
    if c["op"] == "topk":
        ids, weights = mx.moe_topk(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                                   group_score="sum2" if c["sum2"] else "max", renormalize=True, scale=s["scale"], ids=s["ids"], weights=s["weights"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "combine":
        return mx.moe_combine(s["rows"], s["dest"], s["weights"], residual=s["residual"], out=s["y"], status=s["status"])[0]
    act, gate = (None if v == "none" else v for v in (c["act"], c["gate"]))
    if c["op"] == "gemm":
        if c["fmt"] == "nvfp4":
            return mx.gemm_nvfp4(s["x_codes"], s["x_scales"], s["x_g"], s["codes"], s["scales"], s["g"], bias=s["bias"], activation=act, gate=gate,
                                 residual=s["residual"], out=s["y"])
        return mx.gemm(s["x_codes"], s["x_scales"], s["codes"], s["scales"], bias=s["bias"], activation=act, gate=gate, residual=s["residual"], out=s["y"])
    if c["fmt"] == "nvfp4":
        return mx.moe_gemm_nvfp4(s["x_codes"], s["x_scales"], s["x_g"], s["offsets"], s["codes"], s["scales"], s["g"], bias=s["bias"], activation=act,
                                 gate=gate, out=s["y"], status=s["status"])[0]
    return mx.moe_gemm(s["x_codes"], s["x_scales"], s["offsets"], s["codes"], s["scales"], bias=s["bias"], activation=act, gate=gate, out=s["y"],
                       status=s["status"])[0]


def run(state):
    if own:
        return _own(state)
    return {"topk": _plain_topk, "gemm": _plain_gemm, "moe": _plain_moe, "combine": _plain_combine}[state["case"]["op"]](state)


# ------------------------------------------- the definitions in 64 bits
def _exact_elements(codes):
    """E2M1 by its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    e, m = (n >> 1) & 3, n & 1
    a = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    return torch.where(n > 7, -a, a)


def _exact_rows(codes, scales, first, c, cols, g):
    """Rows of codes whose scales begin at row `first` of the tiled buffer, by the layout's formula for each scale's byte."""
    r = torch.arange(first, first + codes.shape[0], device=codes.device).view(-1, 1)
    k = torch.arange(cols, device=codes.device)
    b = scales[((r // 128) * -(-cols // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4].to(torch.int16)
    if c["fmt"] == "mxfp4":
        s = torch.exp2(b.double() - 127)
    else:
        e, m = (b >> 3) & 15, b & 7
        s = torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * torch.exp2((e - 7).double())) / float(g)
    return (_exact_elements(codes).unflatten(-1, (cols, -1)) * s.unsqueeze(-1)).flatten(-2)


def _exact_epilogue(z, c, bias, residual):
    if bias is not None:
        z = z + bias.double()

    def f(v):
        if c["act"] == "silu":
            return v * torch.sigmoid(v)
        return v * torch.special.ndtr(v) if c["act"] == "gelu" else v

    half = z.shape[1] // 2
    if c["gate"] == "first":
        z = f(z[:, :half]) * z[:, half:]
    elif c["gate"] == "second":
        z = z[:, :half] * f(z[:, half:])
    else:
        z = f(z)
    return z if residual is None else z + residual.double()


def _exact_topk(s, c):
    l = s["logits"].double()
    shut = ~torch.isfinite(l)
    l = l.masked_fill(shut, -math.inf)
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, -1), nan=0.0)
    pick = l if s["bias"] is None and not c["sum2"] else score + (0.0 if s["bias"] is None else s["bias"].double())
    pick = pick.masked_fill(shut, -math.inf)

    def best(v, n):
        """The indices of the n largest, one after another, the first of equals; -1 where nothing is left."""
        v, at, out = v.clone(), torch.arange(v.shape[1], device=v.device), []
        for _ in range(n):
            top = v.amax(1, keepdim=True)
            i = torch.where(v == top, at, v.shape[1]).amin(1, keepdim=True)
            out.append(torch.where(top > -math.inf, i, -1))
            v.scatter_(1, i, -math.inf)
        return torch.cat(out, 1)

    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        value = []
        for g in range(c["groups"]):
            part = pick[:, g * size:(g + 1) * size]
            i = best(part, 2 if c["sum2"] and size > 1 else 1)
            v = torch.where(i >= 0, part.gather(1, i.clamp(min=0)), 0.0).sum(1)
            value.append(torch.where(i[:, 0] >= 0, v, -math.inf))
        kept = best(torch.stack(value, 1), c["top_groups"])
        of = torch.arange(c["E"], device=l.device) // size
        pick = torch.where((kept.unsqueeze(2) == of).any(1), pick, -math.inf)
    ids = best(pick, c["k"])
    w = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    total = w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * s["scale"] / torch.where(total > 0, total, 1.0)}


def _exact_gemm(s, c):
    x = _exact_rows(s["x_codes"], s["x_scales"], 0, c, s["cols"], 1.0 if s["x_g"] is None else s["x_g"])
    w = _exact_rows(s["codes"], s["scales"], 0, c, s["cols"], 1.0 if s["g"] is None else s["g"])
    return _exact_epilogue(x @ w.T, c, s["bias"], s["residual"])


def _exact_moe(s, c):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
    per = s["scales"].numel() // c["E"]
    for e in range(c["E"]):
        lo, hi = s["at"][e], s["at"][e + 1]
        if lo < hi:
            x = _exact_rows(s["x_codes"][lo:hi], s["x_scales"], s["padded"][e], c, s["cols"], 1.0 if s["x_g"] is None else s["x_g"][e])
            w = _exact_rows(s["codes"][e], s["scales"][e * per:(e + 1) * per], 0, c, s["cols"], 1.0 if s["g"] is None else s["g"][e])
            y[lo:hi] = _exact_epilogue(x @ w.T, c, None if s["bias"] is None else s["bias"][e], None)
    return y


def _exact_combine(s, c):
    out = []
    for t in range(0, c["T"], 2048):
        dest = s["dest"][t:t + 2048].long()
        w = s["weights"][t:t + 2048].double() * (dest >= 0)
        y = torch.einsum("tj,tjn->tn", w, s["rows"][dest.clamp(min=0)].double())
        out.append(y if s["residual"] is None else y + s["residual"][t:t + 2048].double())
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"topk": _exact_topk, "gemm": _exact_gemm, "moe": _exact_moe, "combine": _exact_combine}[case["op"]](s, case)

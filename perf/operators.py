"""The operators of a decode step on 4-bit weights and a 4-bit cache, as cases to measure.

Four operators, in MXFP4 (32 values to an E8M0 scale) and NVFP4 (16 values to an E4M3 scale and one
float32 global scale), with BF16 or FP16 activations:

matvec     y[t, n] = sum_k x[t, k] * W[n, k], W as packed E2M1 codes and 128x4-tiled scales
moe        the same for every expert's rows of a routed batch (the experts' products)
cache      new keys and values quantized into a paged cache, and a sequence read back from it
attention  one query token per sequence over the paged 4-bit cache

`own` chooses between the plain form (elementary torch operations in float32) and this package's calls.
"""
import math
import random

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a small projection for one token of one user: launch latency
        dict(name="matvec-1tok-small", op="matvec", fmt="mxfp4", dtype="bf16", T=1, N=2048, K=768, f32=False),
        # a square projection of a large hidden size for a few users
        dict(name="matvec-4tok-7168", op="matvec", fmt="nvfp4", dtype="bf16", T=4, N=7168, K=7168, f32=False),
        # the output layer over a vocabulary for a batch, float32 logits
        dict(name="matvec-16tok-vocab", op="matvec", fmt="mxfp4", dtype="f16", T=16, N=64001, K=7168, f32=True),
        # one token's gate and up products: eight of 128 experts
        dict(name="moe-1tok-w13", op="moe", fmt="mxfp4", dtype="bf16", T=1, k=8, E=128, N=1536, K=2048, sorted=False, drop=0.0),
        # a decode batch's gate and up products: nearly every expert has a few rows
        dict(name="moe-64tok-w13", op="moe", fmt="nvfp4", dtype="bf16", T=64, k=8, E=128, N=1536, K=2048, sorted=False, drop=0.0),
        # the down product of a larger batch, rows already in expert order, some routes not dispatched
        dict(name="moe-128tok-w2", op="moe", fmt="mxfp4", dtype="f16", T=128, k=8, E=128, N=2048, K=768, sorted=True, drop=0.1),
        # one new token for each of sixteen sequences, written and read back
        dict(name="cache-16tok", op="cache", fmt="mxfp4", dtype="bf16", T=16, R=16, H=8, D=128, S=16),
        # a chunk of a long prompt written, and the whole prompt so far read back
        dict(name="cache-chunk-8192", op="cache", fmt="mxfp4", dtype="bf16", T=8192, R=32768, H=8, D=128, S=64),
        # odd head count, head size and page size
        dict(name="cache-odd", op="cache", fmt="nvfp4", dtype="f16", T=1000, R=3001, H=5, D=96, S=24),
        # one user, a short context: latency
        dict(name="attention-1seq-short", op="attention", fmt="mxfp4", dtype="bf16", B=1, Hq=64, H=8, D=128, S=16, L=700, window=0),
        # a decode batch of ragged contexts
        dict(name="attention-64seq-8k", op="attention", fmt="mxfp4", dtype="bf16", B=64, Hq=64, H=8, D=128, S=64, L=8192, window=0),
        # one user, a very long context: few rows, a long axis
        dict(name="attention-1seq-128k", op="attention", fmt="nvfp4", dtype="f16", B=1, Hq=64, H=8, D=64, S=32, L=131072, window=0),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("matvec", "moe", "cache", "attention"))
    fmt, dtype = rng.choice(("mxfp4", "nvfp4")), rng.choice(("bf16", "f16"))
    if op == "matvec":
        while True:
            c = dict(op=op, fmt=fmt, dtype=dtype, T=_log(rng, 1, 16), N=_log(rng, 129, 64000), K=_log(rng, 512, 7168, 32), f32=rng.random() < 0.3)
            if c["N"] * c["K"] <= 64001 * 7168:
                return c
    if op == "moe":
        while True:
            c = dict(op=op, fmt=fmt, dtype=dtype, T=_log(rng, 1, 128), k=rng.choice((1, 2, 4, 6, 8)), E=rng.randint(8, 128), N=_log(rng, 256, 4096, 8),
                     K=_log(rng, 512, 4096, 32), sorted=rng.random() < 0.5, drop=rng.choice((0.0, 0.0, 0.2)))
            if c["E"] * c["N"] * c["K"] <= 128 * 1536 * 2048:
                return c
    if op == "cache":
        while True:
            c = dict(op=op, fmt=fmt, dtype=dtype, T=_log(rng, 1, 8192), R=_log(rng, 1, 32768), H=rng.randint(1, 16), D=rng.choice((64, 96, 128, 192, 256)),
                     S=_log(rng, 8, 128))
            if (c["T"] + c["R"]) * c["H"] * c["D"] <= 40960 * 1024:
                return c
    while True:
        H = rng.choice((1, 2, 4, 5, 8))
        c = dict(op=op, fmt=fmt, dtype=dtype, B=_log(rng, 1, 64), Hq=H * rng.choice((1, 4, 7, 8, 16)), H=H, D=rng.choice((64, 96, 128, 256)), S=_log(rng, 8, 128),
                 L=_log(rng, 64, 131072), window=rng.choice((0, 0, 0, 1000)))
        if c["B"] * c["L"] * c["H"] * c["D"] <= 64 * 8192 * 8 * 128 and c["B"] * c["L"] * c["Hq"] <= 64 * 8192 * 64:
            return c


def _lengths(c):
    """The contexts' lengths, from half of L to L: the case alone says them."""
    rng = random.Random("%d %d %d" % (c["B"], c["L"], c["S"]))
    return [c["L"] if b == 0 else rng.randint(c["L"] // 2, c["L"]) for b in range(c["B"])]


def work(c):
    per = 0.5 + (1 / 32 if c["fmt"] == "mxfp4" else 1 / 16)   # bytes of a 4-bit value and its share of a scale
    if c["op"] == "matvec":
        return {"bytes": c["N"] * c["K"] * per + 2 * c["T"] * c["K"] + (4 if c["f32"] else 2) * c["T"] * c["N"], "flops": 2 * c["T"] * c["N"] * c["K"]}
    if c["op"] == "moe":
        top_k = min(c["k"], c["E"])
        rows = c["T"] * top_k * (1 - c["drop"])
        used = c["E"] * (1 - (1 - top_k * (1 - c["drop"]) / c["E"]) ** c["T"])     # experts that a uniform routing reaches
        x = rows if c["sorted"] else c["T"]
        return {"bytes": used * c["N"] * c["K"] * per + 2 * x * c["K"] + 2 * rows * c["N"], "flops": 2 * rows * c["N"] * c["K"]}
    if c["op"] == "cache":
        return {"bytes": (c["T"] + c["R"]) * 2 * c["H"] * c["D"] * (2 + per), "flops": 0}
    n = sum(min(v, c["window"]) if c["window"] else v for v in _lengths(c))
    return {"bytes": n * c["H"] * c["D"] * 2 * per + 4 * c["B"] * c["Hq"] * c["D"] + 4 * c["B"] * c["Hq"], "flops": 4 * n * c["Hq"] * c["D"]}


# ------------------------------------------------------- the plain forms
def _table(device):
    """Both values of each code byte, the even element first."""
    v = torch.tensor(_E2M1 + tuple(-a for a in _E2M1), device=device)
    i = torch.arange(256, device=device)
    return torch.stack((v[i % 16], v[i // 16]), 1)


def _decode(codes, table):
    """Packed codes [..., n] -> float32 E2M1 values [..., 2n]."""
    return table[codes.int()].flatten(-2)


def _scale_values(scales, fmt):
    """Scale bytes -> float32: 2^(s - 127), or the E4M3 value."""
    if fmt == "nvfp4":
        return scales.view(torch.float8_e4m3fn).float()
    s = scales.int()
    v = torch.where(s == 0, 1 << 22, s << 23).view(torch.float32)
    return torch.where(s == 255, math.nan, v)


def _untile(scales, rows, cols):
    """128x4-tiled scale bytes [..., bytes] -> [..., rows, cols]."""
    mt, kt = -(-rows // 128), -(-cols // 4)
    t = scales.view(*scales.shape[:-1], mt, kt, 32, 4, 4)
    n = t.dim()
    t = t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1)
    return t.reshape(*scales.shape[:-1], mt * 128, kt * 4)[..., :rows, :cols]


def _tile(flat):
    """[..., rows, cols] scale bytes -> 128x4-tiled bytes [..., bytes], padded with zeros."""
    rows, cols = flat.shape[-2:]
    mt, kt = -(-rows // 128), -(-cols // 4)
    p = torch.zeros(*flat.shape[:-2], mt * 128, kt * 4, dtype=torch.uint8, device=flat.device)
    p[..., :rows, :cols] = flat
    t = p.view(*flat.shape[:-2], mt, 4, 32, kt, 4)
    n = t.dim()
    t = t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1)
    return t.reshape(*flat.shape[:-2], -1)


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
    """float32 values of codes [..., n/2] with flat scale bytes."""
    s = _scale_values(scales, fmt)
    v = _decode(codes, table).unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)
    return (v if fmt == "mxfp4" else v * (1.0 / g)).flatten(-2)


def _plain_matvec(s):
    c = s["case"]
    w = _values(s["codes"], _untile(s["scales"], c["N"], s["cols"]), c["fmt"], s["g"], s["e2m1"])
    return (s["x"].float() @ w.T).to(s["y"].dtype)


def _plain_moe(s):
    c = s["case"]
    E, T = c["E"], c["T"]
    g = s["g"].view(E, 1, 1) if c["fmt"] == "nvfp4" else None
    w = _decode(s["codes"], s["e2m1"]).unflatten(-1, (s["cols"], -1)) * _scale_values(_untile(s["scales"].view(E, -1), c["N"], s["cols"]), c["fmt"]).unsqueeze(-1)
    w = w.flatten(-2) if g is None else w.flatten(-2) * (1.0 / g)
    rows = s["y"].shape[0]
    r = torch.arange(rows, device=w.device)
    e = torch.searchsorted(s["offsets"], r, right=True, out_int32=True).long() - 1      # E for the rows that no route fills
    at = torch.where(e < E, r - s["offsets"][e.clamp(max=E)], 0)
    x = s["x"] if c["sorted"] else s["x"][torch.where(e < E, s["row_index"], 0).long()]
    padded = torch.zeros(E + 1, T, c["K"], device=w.device)
    padded[e, at] = x.float()
    y = torch.bmm(padded[:E], w.transpose(1, 2))
    y = torch.where((e < E).unsqueeze(1), y[e.clamp(max=E - 1), at], 0.0)
    return y.to(s["y"].dtype)


def _places(slots, S):
    return slots.long() // S, slots.long() % S


def _plain_cache(s):
    c = s["case"]
    out = {}
    for part in ("k", "v"):
        codes, scales = s[part + "_codes"], s[part + "_scales"]
        g = s["g_" + part]
        new_codes, new_scales = _quantize(s[part], c["fmt"], g)
        page, at = _places(s["slots"], c["S"])
        codes[page, :, at] = new_codes
        scales[page, :, at] = new_scales
        page, at = _places(s["read"], c["S"])
        out[part] = _values(codes[page, :, at], scales[page, :, at], c["fmt"], g, s["e2m1"]).to(s["k"].dtype)
    return out


def _plain_attention(s):
    c = s["case"]
    B, H, D, G = c["B"], c["H"], c["D"], c["Hq"] // c["H"]
    n = s["tokens"]
    table = s["table"].long()

    def values(part):
        codes, scales = (s[part + t][table].transpose(2, 3).flatten(1, 2) for t in ("_codes", "_scales"))     # [B, tokens, H, ...]
        return _values(codes, scales, c["fmt"], s["g_" + part], s["e2m1"]).transpose(1, 2)                              # [B, H, tokens, D]

    j = torch.arange(n, device=table.device)
    size = s["lens"].view(B, 1)
    seen = (j < size) & (j >= (size - c["window"] if c["window"] else 0))
    a = s["q"].float().view(B, H, G, D) @ values("k").transpose(2, 3) * s["scale"]
    a = torch.where(seen.view(B, 1, 1, n), a, -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top > -math.inf, top, 0.0))
    z = p.sum(-1, keepdim=True)
    o = p @ values("v") / torch.where(z > 0, z, 1.0)
    return {"o": o.reshape(B, c["Hq"], D).to(s["q"].dtype), "lse": (top + torch.log(z)).reshape(B, c["Hq"])}


# --------------------------------------------------------------- inputs
def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _weights(gen, c, rows, device, experts=None):
    """Quantized N(0, 0.02^2) weights: codes and tiled scales, drawn in pieces."""
    K, fmt = c["K"], c["fmt"]
    amax = 0.12
    g = None if fmt == "mxfp4" else torch.full((experts or 1,), 448.0 * 6.0 / amax, device=device)
    if g is not None and experts:
        g = g * (1.0 + torch.rand(experts, device=device, generator=gen))
    codes, flat = [], []
    total = rows * (experts or 1)
    step = rows if experts else 16384
    for k, r in enumerate(range(0, total, step)):
        w = (torch.randn(min(step, total - r), K, device=device, generator=gen) * 0.02).bfloat16()
        q, s = _quantize(w, fmt, None if g is None else g[k if experts else 0])
        codes.append(q)
        flat.append(s)
    codes, flat = torch.cat(codes), torch.cat(flat)
    cols = flat.shape[-1]
    if experts:
        codes, flat = codes.view(experts, rows, K // 2), flat.view(experts, rows, cols)
    return codes, _tile(flat).reshape(-1), g, cols


def _prepare_matvec(c, seed, device):
    gen = _generator(seed, device)
    codes, scales, g, cols = _weights(gen, c, c["N"], device)
    x = torch.randn(c["T"], c["K"], device=device, generator=gen).to(_TYPES[c["dtype"]])
    y = torch.empty(c["T"], c["N"], device=device, dtype=torch.float32 if c["f32"] else x.dtype)
    return dict(codes=codes, scales=scales, g=g, cols=cols, x=x, y=y)


def _prepare_moe(c, seed, device):
    gen = _generator(seed, device)
    E, T, k = c["E"], c["T"], min(c["k"], c["E"])
    codes, scales, g, cols = _weights(gen, c, c["N"], device, experts=E)
    ids = torch.rand(T, E, device=device, generator=gen).topk(k, 1).indices
    ids[torch.rand(T, k, device=device, generator=gen) < c["drop"]] = E            # not dispatched: sorted to the end
    ids, order = ids.reshape(-1).sort(stable=True)
    offsets = torch.searchsorted(ids, torch.arange(E + 1, device=device)).to(torch.int32)
    row_index = (order // k).to(torch.int32)
    x = torch.randn(T * k if c["sorted"] else T, c["K"], device=device, generator=gen).to(_TYPES[c["dtype"]])
    y = torch.zeros(T * k, c["N"], device=device, dtype=x.dtype)
    status = torch.zeros(1, device=device, dtype=torch.int32)
    return dict(codes=codes, scales=scales, g=g, cols=cols, x=x, y=y, offsets=offsets, row_index=row_index, status=status)


def _cache(gen, c, pages, device):
    """A filled cache: [pages, H, S, ...] codes and scales of N(0, 1) keys and values."""
    H, S, D, fmt = c["H"], c["S"], c["D"], c["fmt"]
    s = {"g_k": None, "g_v": None}
    if fmt == "nvfp4":
        s["g_k"], s["g_v"] = (torch.full((1,), 448.0 * 6.0 / a, device=device) for a in (8.0, 6.5))
    for part in ("k", "v"):
        codes = torch.empty(pages, H, S, D // 2, dtype=torch.uint8, device=device)
        scales = torch.empty(pages, H, S, D // (32 if fmt == "mxfp4" else 16), dtype=torch.uint8, device=device)
        step = max(1, (1 << 25) // (H * S * D))
        for p in range(0, pages, step):
            x = torch.randn(min(step, pages - p), H, S, D, device=device, generator=gen).to(_TYPES[c["dtype"]])
            codes[p:p + step], scales[p:p + step] = _quantize(x, fmt, s["g_" + part])
        s[part + "_codes"], s[part + "_scales"] = codes, scales
    return s


def _prepare_cache(c, seed, device):
    gen = _generator(seed, device)
    T, R, H, D, S = c["T"], c["R"], c["H"], c["D"], c["S"]
    pages = -(-max(T, R) // S) + 3
    s = _cache(gen, c, pages, device)
    kv = torch.randn(T, 2, H, D, device=device, generator=gen).to(_TYPES[c["dtype"]])     # the two halves of one projection's output
    order = torch.randperm(pages, device=device, generator=gen)[:-(-max(T, R) // S)]
    at = torch.arange(max(T, R), device=device)
    where = (order[at // S] * S + at % S).to(torch.int32)
    s.update(k=kv[:, 0], v=kv[:, 1], slots=where[-T:].clone(), read=where[:R].clone())
    s.update(k_out=torch.empty(R, H, D, device=device, dtype=kv.dtype), v_out=torch.empty(R, H, D, device=device, dtype=kv.dtype))
    s.update(status=torch.zeros(1, device=device, dtype=torch.int32))
    return s


def _prepare_attention(c, seed, device):
    gen = _generator(seed, device)
    B, Hq, H, D, S = c["B"], c["Hq"], c["H"], c["D"], c["S"]
    per = -(-c["L"] // S)
    s = _cache(gen, c, B * per, device)
    s["table"] = torch.randperm(B * per, device=device, generator=gen).view(B, per).to(torch.int32)
    s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=device)
    s["q"] = torch.randn(B, Hq, D, device=device, generator=gen).to(_TYPES[c["dtype"]])
    s.update(scale=D ** -0.5, tokens=per * S, o=torch.empty_like(s["q"]), lse=torch.empty(B, Hq, device=device), status=torch.zeros(1, device=device, dtype=torch.int32))
    return s


def prepare(case, seed):
    make = {"matvec": _prepare_matvec, "moe": _prepare_moe, "cache": _prepare_cache, "attention": _prepare_attention}[case["op"]]
    device = torch.device("cuda")
    return dict(make(case, seed, device), e2m1=_table(device), case=case)


# ----------------------------------------------------------- one pass
def _own(s):
    import mxfp4_block_quantization_gb300 as mx

    op, nv = s["case"]["op"], s["case"]["fmt"] == "nvfp4"
    if op == "matvec":
        return mx.matvec_nvfp4(s["x"], s["codes"], s["scales"], s["g"], out=s["y"]) if nv else mx.matvec(s["x"], s["codes"], s["scales"], out=s["y"])
    if op == "moe":
        rows = None if s["case"]["sorted"] else s["row_index"]
        if nv:
            return mx.moe_matvec_nvfp4(s["x"], rows, s["offsets"], s["codes"], s["scales"], s["g"], out=s["y"], status=s["status"])[0]
        return mx.moe_matvec(s["x"], rows, s["offsets"], s["codes"], s["scales"], out=s["y"], status=s["status"])[0]
    cache = mx.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["g_k"], s["g_v"])
    if op == "cache":
        mx.cache_write(s["k"], s["v"], s["slots"], cache, status=s["status"])
        k, v, _ = mx.cache_read(cache, s["read"], k_out=s["k_out"], v_out=s["v_out"], status=s["status"])
        return {"k": k, "v": v}
    o, lse, _ = mx.cache_attention(s["q"], cache, s["table"], s["lens"], s["scale"], window=s["case"]["window"], out=s["o"], lse=s["lse"], status=s["status"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"matvec": _plain_matvec, "moe": _plain_moe, "cache": _plain_cache, "attention": _plain_attention}[state["case"]["op"]](state)


# ------------------------------------------- the definitions in 64 bits
def _exact_elements(codes):
    """E2M1 by its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    e, m = (n >> 1) & 3, n & 1
    a = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    return torch.where(n > 7, -a, a)


def _exact_scale(b, fmt):
    """E8M0 and E4M3 bytes by their fields."""
    i = b.to(torch.int16)
    if fmt == "mxfp4":
        return torch.exp2(i.double() - 127)
    e, m = (i >> 3) & 15, i & 7
    return torch.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * torch.exp2((e - 7).double()))


def _exact_rows(codes, scales, fmt, g):
    s = _exact_scale(scales, fmt)
    v = (_exact_elements(codes).unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)
    return v if fmt == "mxfp4" else v / float(g)


def _exact_untiled(scales, rows, cols):
    """The scale of row r and column c, by the layout's formula for its byte."""
    r = torch.arange(rows, device=scales.device).view(-1, 1)
    c = torch.arange(cols, device=scales.device)
    return scales[((r // 128) * -(-cols // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]


def _exact_quantized(x, fmt, g):
    """The values that the quantizers' rules give, with logarithms and distances in place of bits and thresholds."""
    block = 32 if fmt == "mxfp4" else 16
    v = x.double().unflatten(-1, (-1, block))
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        m, e = torch.frexp(top)                                # top = m 2^e with m in [0.5, 1)
        s = (e - 1 + 127 + (m * 2 >= 1.75).int()).clamp(min=0)
        s = torch.where(s > 2, s - 2, 0)
        scale = torch.where(s > 0, torch.exp2(s.double() - 127), 0.0)
        a = v.abs() / torch.where(scale > 0, scale, 1.0)
    else:                                                             # the roundings to float32 are part of the rule
        sf = ((top.float() / 6.0) * g).clamp(max=448.0).double()
        step = torch.exp2(torch.floor(torch.log2(sf.clamp(min=2.0 ** -6))) - 3)
        byte = torch.round(sf / step) * step                          # torch.round: ties to even
        scale = byte / float(g)
        a = (v.abs().float() * (float(g) / torch.where(byte > 0, byte, 1.0)).float()).double()
    grid = torch.tensor(_E2M1, device=x.device, dtype=torch.float64)
    a = torch.where(scale > 0, a, 0.0)
    best, value = torch.full_like(a, math.inf), torch.zeros_like(a)
    for i in (0, 2, 4, 6, 1, 3, 5, 7):                           # the even codes first: they win the ties
        d = (a - grid[i]).abs()
        value = torch.where(d < best, grid[i], value)
        best = torch.minimum(best, d)
    return (torch.sign(v) * value * scale).flatten(-2)


def _exact_matvec(s, c):
    out = []
    flat = _exact_untiled(s["scales"], c["N"], s["cols"])
    g = 1.0 if s["g"] is None else s["g"]
    for r in range(0, c["N"], 8192):
        out.append(s["x"].double() @ _exact_rows(s["codes"][r:r + 8192], flat[r:r + 8192], c["fmt"], g).T)
    return torch.cat(out, 1)


def _exact_moe(s, c):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
    at, per = s["offsets"].tolist(), s["scales"].numel() // c["E"]
    for e in range(c["E"]):
        lo, hi = at[e], at[e + 1]
        if lo < hi:
            w = _exact_rows(s["codes"][e], _exact_untiled(s["scales"][e * per:(e + 1) * per], c["N"], s["cols"]), c["fmt"], 1.0 if s["g"] is None else s["g"][e])
            x = s["x"][lo:hi] if c["sorted"] else s["x"][s["row_index"][lo:hi].long()]
            y[lo:hi] = x.double() @ w.T
    return y


def _exact_cache(s, c):
    out = {}
    for part in ("k", "v"):
        old = _exact_rows(s[part + "_codes"], s[part + "_scales"], c["fmt"], 1.0 if s["g_" + part] is None else s["g_" + part])
        old = old.transpose(1, 2).flatten(0, 1)                   # by slot
        old[s["slots"].long()] = _exact_quantized(s[part], c["fmt"], s["g_" + part])
        out[part] = old[s["read"].long()]
    return out


def _exact_attention(s, c):
    G = c["Hq"] // c["H"]
    o, lse = [], []
    for b, size in enumerate(s["lens"].tolist()):
        lo = max(0, size - c["window"]) if c["window"] else 0
        pages = s["table"][b].long()

        def rows(part):
            v = _exact_rows(s[part + "_codes"][pages], s[part + "_scales"][pages], c["fmt"], 1.0 if s["g_" + part] is None else s["g_" + part])
            return v.transpose(0, 1).flatten(1, 2)[:, lo:size]       # [H, tokens, D]

        a = s["scale"] * torch.einsum("hgd,htd->hgt", s["q"][b].double().view(c["H"], G, -1), rows("k"))
        lse.append(torch.logsumexp(a, -1).reshape(-1))
        o.append(torch.einsum("hgt,htd->hgd", torch.softmax(a, -1), rows("v")).reshape(c["Hq"], -1))
    return {"o": torch.stack(o), "lse": torch.stack(lse)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"matvec": _exact_matvec, "moe": _exact_moe, "cache": _exact_cache, "attention": _exact_attention}[case["op"]](s, case)

"""Plain 64-bit forms of a layer's operators over many tokens (the router's
choice, products of 4-bit activations with 4-bit weights, the experts' rows back
to their tokens), from their definitions, and the error bounds their float32
kernels are held to.  Any device."""
import math

import torch

import decode_reference as R


# ------------------------------------------------------------- the router
def topk(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max",
         renormalize=True, scale=1.0):
    """(ids, weights float64, the weights' bound) of logits [T, E]."""
    l = logits.double()
    T, E = l.shape
    b = torch.zeros(E, dtype=torch.float64, device=l.device) if bias is None else bias.double()
    live = torch.isfinite(l)
    if score == "sigmoid":
        s = torch.where(live, torch.sigmoid(l), 0.0)
    else:
        s = torch.nan_to_num(torch.softmax(l.masked_fill(~live, -math.inf), -1), nan=0.0)
    live = live & torch.isfinite(b)
    logits_decide = bias is None and (groups == 1 or group_score == "max")
    pick = torch.where(live, l if logits_decide else s + b, -math.inf)
    ids = torch.full((T, top_k), -1, dtype=torch.int64)
    size = E // groups
    for t, row in enumerate(pick.tolist()):
        kept = range(groups)
        if groups > 1:
            value = []
            for g in range(groups):
                best = sorted((v for v in row[g * size:(g + 1) * size] if v > -math.inf), reverse=True)
                n = 2 if group_score == "sum2" else 1
                value.append(sum(best[:n]) if best else -math.inf)
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        open_ = [e for e in range(E) if row[e] > -math.inf and e // size in kept]
        for j, e in enumerate(sorted(open_, key=lambda e: (-row[e], e))[:top_k]):
            ids[t, j] = e
    ids = ids.to(l.device)
    there = ids >= 0
    at = ids.clamp(min=0)
    w = torch.where(there, s.gather(1, at), 0.0)
    chosen = torch.where(there, l.gather(1, at), 0.0)
    if renormalize:
        # of the scores' logarithms, so that none vanishes
        log = torch.nn.functional.logsigmoid(chosen) if score == "sigmoid" else chosen
        w = torch.nan_to_num(torch.softmax(log.masked_fill(~there, -math.inf), -1), nan=0.0)
    # e^x is off by 2^-22 and by 2^-24 |x| for its argument; sums of up to 8192
    # terms in lanes and a tree by 2^-16, of the chosen 32 by 2^-21
    far = torch.where(live, l, 0.0).abs().amax(-1, keepdim=True) + chosen.abs()
    off = 2.0 ** -19 + 2.0 ** -22 * far + (0.0 if renormalize or score == "sigmoid" else E * 2.0 ** -28)
    w = w * scale
    return ids.to(torch.int32), w, w.abs() * off + 2.0 ** -140


# ------------------------------------------------------------- the products
def activated(z, act):
    """act(z) in float64."""
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def gemm(x, w, dtype, bias=None, act=None, gate=None, residual=None):
    """(y, bound) of x [T, K] times the transpose of w [N, K] (float64).

    Bound: each of K products and additions of the sum in float32 may be off by
    2^-23 of the terms' magnitudes (an addition that truncates), the scaling and
    the bias by 2^-23 of what they make.  No activation here is steeper than
    1.13; its own float32 steps leave 2^-20 of |z|."""
    K = x.shape[1]
    z = x @ w.T
    off = (K + 8) * 2.0 ** -23 * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + bias.double()
        off = off + 2.0 ** -23 * (z.abs() + bias.double().abs())

    def act_of(v, o):
        if act is None:
            return v, o
        return activated(v, act), 1.13 * o + 2.0 ** -20 * v.abs()

    if gate is None:
        y, off = act_of(z, off)
    else:
        h = z.shape[1] // 2
        g, u = ((z[:, :h], off[:, :h]), (z[:, h:], off[:, h:]))
        if gate == "second":
            g, u = u, g
        (a, da), (b, db) = act_of(*g), u
        y = a * b
        off = da * b.abs() + a.abs() * db + da * db + 2.0 ** -23 * y.abs()
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -23 * (y.abs() + residual.double().abs())
    return y, off + R.unit(dtype) * (y.abs() + off) + R.smallest(dtype)


def close(got, want, bound):
    """R.close for values that may be too large for the type of `got`: rounding to
    nearest gives infinity from its largest value and half a step on, so there an
    infinity of the sign is asked for, and either where the bound spans that edge."""
    edge = {torch.float16: 65520.0, torch.bfloat16: (2 - 2.0 ** -8) * 2.0 ** 127}[got.dtype]
    inf = torch.where(want > 0, math.inf, -math.inf).to(torch.float64)
    out = torch.where(want.abs() - bound >= edge, inf, want)
    either = (want.abs() + bound >= edge) & (got.double() == inf)
    R.close(got, torch.where(either, inf, out), bound)


# ------------------------------------------------------------- the way back
def combine(rows, dest, weights, dtype, residual=None):
    """(y, bound): top_k products and additions in float32, each off by 2^-24 of
    its partial sum at most, which the magnitudes' sum bounds; one rounding."""
    there = (dest >= 0) & (dest < rows.shape[0])
    T, k = dest.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    mass = torch.zeros_like(y)
    if residual is not None:
        y, mass = residual.double(), residual.double().abs()
    for j in range(k):
        if rows.shape[0]:
            term = rows.double()[dest[:, j].long().clamp(0, rows.shape[0] - 1)]
            term = torch.where(there[:, j:j + 1], weights[:, j:j + 1].double() * term, 0.0)
            y, mass = y + term, mass + term.abs()
    off = (k + 1) * 2.0 ** -23 * mass
    return y, off + R.unit(dtype) * (y.abs() + off) + R.smallest(dtype)

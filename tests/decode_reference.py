"""Plain 64-bit forms of the decode-step operators, from their definitions
(products with 4-bit weights, the paged 4-bit cache, attention over it), and
the error bounds their float32 kernels are held to.  Any device."""
import math

import torch

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def elements(codes):
    """Packed codes [..., n] -> the E2M1 values [..., 2n], float64."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64,
                         device=codes.device)
    return table[torch.stack((codes & 15, codes >> 4), -1).long()].flatten(-2)


def scale_values(b, nvfp4):
    """Scale bytes -> float64: 2^(s-127) (255: NaN), or the E4M3 value."""
    if nvfp4:
        return b.view(torch.float8_e4m3fn).double()
    i = b.double()
    return torch.where(i == 255, math.nan, torch.exp2(i - 127))


def untile(scales, rows, cols):
    """Tiled scale bytes -> [rows, cols], by the layout's formula."""
    r = torch.arange(rows, device=scales.device).view(-1, 1)
    c = torch.arange(cols, device=scales.device)
    return scales[((r // 128) * -(-cols // 4) + c // 4) * 512 + (r % 32) * 16 +
                  (r % 128) // 32 * 4 + c % 4]


def rows_of(codes, flat_scales, nvfp4, g=1.0):
    """The values of codes [..., n/2] with flat scale bytes, float64."""
    s = scale_values(flat_scales, nvfp4)
    v = elements(codes)
    if v.numel():
        v = (v.unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)
    return v / float(g) if nvfp4 else v


def weights(codes, scales, nvfp4, g=1.0):
    """[N, K] float64 of packed codes [N, K/2] and tiled scales."""
    N, K = codes.shape[0], codes.shape[1] * 2
    return rows_of(codes, untile(scales, N, K // (16 if nvfp4 else 32)), nvfp4, g)


def unit(dtype):
    """Largest relative error of rounding to ``dtype`` (half a spacing at 1)."""
    return {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]


def smallest(dtype):
    """Half the spacing of ``dtype``'s subnormals."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25,
            torch.float32: 2.0 ** -150}[dtype]


def product(x, w, dtype):
    """(y, bound) of x [T, K] times the transpose of w [N, K].

    Bound: each of K products and additions in float32 may be off by 2^-23 of
    the terms' sum of magnitudes (an addition that truncates), the values of x
    by 2^-40 of the largest of their block of 32 and the final rounding by
    half a spacing of the output's type."""
    x = x.double()
    K = x.shape[1]
    y = x @ w.T
    block = torch.zeros_like(x)
    if K:
        pad = torch.nn.functional.pad(x.abs(), (0, -K % 32)).unflatten(1, (-1, 32))
        block = pad.amax(-1, keepdim=True).expand_as(pad).flatten(1)[:, :K]
    mass = x.abs() @ w.abs().T
    off = (K + 8) * 2.0 ** -23 * mass + 2.0 ** -40 * (block @ w.abs().T)
    return y, off + unit(dtype) * (y.abs() + off) + smallest(dtype)


def attention(q, k, v, scale, dtype):
    """(o, o's bound, lse, lse's bound) of q [heads, D] over k, v [n, D] of one
    kv head.

    Bound: a score is off by 2^-23 (D + 8) of its terms' magnitudes, which
    moves its weight by twice that; a weight may be rounded to 11 bits
    (2^-11), or lost under 2^-24 of the largest scale of its tile (so 2^-24 of
    the largest value); the sums of n terms by 2^-23 each and exp by 2^-20."""
    q, k, v = q.double(), k.double(), v.double()
    n, D = k.shape
    if n == 0:
        z = torch.zeros_like(q)
        inf = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
        return z, z, inf, torch.zeros_like(inf)
    a = scale * (q @ k.T)
    d = abs(scale) * (D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T)
    p = torch.softmax(a, -1)
    o = p @ v
    mass = p @ v.abs()
    rel = 2.0 ** -10 + 4 * d.amax(-1, keepdim=True) + n * 2.0 ** -22 + 2.0 ** -19
    off = rel * mass + 2.0 ** -23 * v.abs().amax()
    lse = torch.logsumexp(a, -1)
    lse_off = d.amax(-1) + n * 2.0 ** -22 + 2.0 ** -19 + 2.0 ** -22 * lse.abs()
    return o, off + unit(dtype) * (o.abs() + off) + smallest(dtype), lse, lse_off


def close(got, want, bound):
    """Every element within its bound, NaN and infinities at the same places."""
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN at other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = ((got - want).abs() - bound)[fine]
    if off.numel():
        worst = off.argmax()
        assert off[worst] <= 0, (f"off by {(got - want).abs()[fine][worst]:.3g}, bound "
                                 f"{bound.expand_as(want)[fine][worst]:.3g}, value "
                                 f"{want[fine][worst]:.3g}")

"""Error bounds of the decode operators that grow with the square root of a sum's
length, for data without a common sign: a lost block of 32 elements or positions
is far outside them, where a bound on every term's worst rounding lets it pass.
Any device."""
import torch

import decode_reference as R


def product(x, w, dtype):
    """(y, bound) of x [T, K] times the transpose of w [N, K], both of random signs.

    A partial sum of k terms of random signs is within 6 sqrt(k) of their root mean
    square s.  The tensor cores add 16 terms at a time with an error of up to 2^-22
    of the partial sum, and float32 adds each block of 32 at 2^-24 of it: K / 16
    additions of at most 2^-21 each.  The bound is their sum's."""
    x = x.double()
    K = x.shape[1]
    y = x @ w.T
    s = ((x * x) @ (w * w).T / K).sqrt()
    off = (K / 16 + 8) * 2.0 ** -21 * 6 * K ** 0.5 * s
    return y, off + R.unit(dtype) * (y.abs() + off) + R.smallest(dtype)


def attention(q, k, v, scale, dtype):
    """(o, o's bound) of q [heads, D] over k, v [n, D], v of random signs.

    S = sqrt(sum p^2 v^2) is the spread of o.  Weights rounded to 11 bits, with and
    without v's scale, move o by 2^-11 S or less in the root mean square (8 of it are
    allowed); scores that are off by d move it by 4 d S; and a sum of at most 2048 products of
    16 positions (of longer contexts a warp has a part), by 2^-21 of partial sums
    within 6 S each."""
    q, k, v = q.double(), k.double(), v.double()
    n, D = k.shape
    a = scale * (q @ k.T)
    d = abs(scale) * (D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T)
    p = torch.softmax(a, -1)
    o = p @ v
    spread = ((p * p) @ (v * v)).sqrt()
    off = (8 * 2.0 ** -11 + 4 * d.amax(-1, keepdim=True) + min(n / 16, 2048) * 2.0 ** -21 * 6) * spread
    return o, off + R.unit(dtype) * (o.abs() + off) + R.smallest(dtype)

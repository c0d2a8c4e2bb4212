"""Attention over the paged 4-bit cache where few bits decide, and near the ends of
float32."""
import math

import pytest
import torch

import decode_reference as R
from test_gpu_attention_split import with_room
from test_gpu_cache import BF16, F16, filled, make_cache, mx, rand, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def contents(c, pages, n):
    """The keys and values [heads, n, head_dim] of the pages' first n positions, float64."""
    nvfp4 = c.k_global is not None

    def rows(codes, scales, g):
        x = R.rows_of(codes[pages], scales[pages], nvfp4, 1.0 if g is None else g)
        return x.transpose(0, 1).flatten(1, 2)[:, :n]

    return rows(c.k_codes, c.k_scales, c.k_global), rows(c.v_codes, c.v_scales, c.v_global)


@pytest.mark.parametrize("gap", [8.3, 16.4, 20.3, 22.6, 24.4])
@pytest.mark.parametrize("n,room", [(32, False), (250, False), (250, True), (1700, False), (1700, True)])
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_tail_beside_a_dominant_position(mx, gap, n, room, nvfp4, dtype):  # noqa: F811
    """One position's weight is 2^gap times the others' and its value is zero, as a
    sink of attention has it: the output is the others'.

    Bound: a weight is rounded to 11 bits twice (with its value's scale), and no
    finer than 2^-36 of the largest weight, times the largest value."""
    S, D = 16, 64
    pages = -(-n // S)
    c = make_cache(mx, pages, S, 1, D, nvfp4)
    k, v = torch.zeros((n, 1, D), dtype=dtype, device="cuda"), rand((n, 1, D), n, dtype)
    k[3, 0, 0], v[3] = 4.0, 0.0
    mx.cache_write(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), c)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    q = torch.zeros((1, 3, D), dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([1.0, 0.5, 2.0])
    scale = gap * math.log(2.0) / 4.0
    o, lse, _ = mx.cache_attention(q, c, with_room(table, S) if room else table,
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), scale)
    kd, vd = contents(c, table[0].long(), n)
    a = scale * (q[0].double() @ kd[0].T)
    p = torch.softmax(a, -1)
    want = p @ vd[0]
    off = (2.0 ** -10 + 2.0 ** -18) * (p @ vd[0].abs()) + n * 2.0 ** -36 * vd.abs().amax()
    keep = [0, 1] if gap > 12 else [0, 1, 2]             # 2.0: twice the gap
    R.close(o[0, keep], want[keep], (off + R.unit(dtype) * (want.abs() + off) + R.smallest(dtype))[keep])
    R.close(lse[0], torch.logsumexp(a, -1), 2.0 ** -18 + 2.0 ** -22 * a.abs().amax(-1))


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("v_global", [1e36, -3e38, 1e-30])
def test_global_scale_of_values_near_the_range(mx, v_global, room):  # noqa: F811
    """The sum of the weights times the values' global scale is past float32."""
    n, S, D = 1000, 16, 64
    c = filled(mx, 64, S, 1, D, True, 6)
    c.v_scales.fill_(0x38)                                           # 1.0
    c.v_codes.fill_(0x77)                                            # 6.0 everywhere
    c = c._replace(v_global=torch.tensor([v_global], device="cuda"))
    table = tables(1, 63, 64, 1)
    q = rand((1, 4, D), 5)
    o, _, _ = mx.cache_attention(q, c, with_room(table, S) if room else table,
                                 torch.tensor([n], dtype=torch.int32, device="cuda"), 0.01)
    want = torch.full((1, 4, D), 6.0 / v_global, dtype=torch.float64, device="cuda")
    R.close(o, want, 2.0 ** -7 * want.abs() + R.smallest(BF16))


def key_scales(c, low, high, seed):
    """Random E8M0 bytes in [low, high] for the keys."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c.k_scales.copy_(torch.randint(low, high + 1, c.k_scales.shape, device="cuda", generator=gen).to(torch.uint8))


def check_scores(mx, q, c, n, scale, room, S=16):
    table = tables(1, -(-n // S), c.k_codes.shape[0], 1)
    o, lse, _ = mx.cache_attention(q, c, with_room(table, S) if room else table,
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), scale)
    k, v = contents(c, table[0].long(), n)
    G = q.shape[1] // k.shape[0]
    for h in range(k.shape[0]):
        want, bound, wl, bl = R.attention(q[0, h * G:(h + 1) * G], k[h], v[h], scale, q.dtype)
        R.close(o[0, h * G:(h + 1) * G], want, bound)
        R.close(lse[0, h * G:(h + 1) * G], wl, bl)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("scale", [0.0, 1e-39, -3e-45, 2.0 ** -104])
def test_vanishing_scales_beside_large_keys(mx, scale, room):  # noqa: F811
    c = filled(mx, 20, 16, 2, 64, False, 6)
    key_scales(c, 127 + 100, 127 + 103, 1)
    check_scores(mx, rand((1, 8, 64), 5), c, 300, scale, room)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("key,query", [(110, 0), (118, -20), (123, -100), (60, 60), (-120, 0), (-126, 20), (-60, -60)])
def test_keys_and_queries_near_the_range(mx, key, query, room):  # noqa: F811
    """Keys of up to 2^125 and down to 2^-127: the scores are of ordinary size
    after the softmax's scale."""
    c = filled(mx, 20, 16, 2, 64, False, 6)
    key_scales(c, max(127 + key - 1, 0), 127 + key + 1, 2)
    q = (rand((1, 8, 64), 5).float() * 2.0 ** query).to(BF16)
    check_scores(mx, q, c, 300, 0.1 * 2.0 ** -max(min(key + query, 125), -125), room)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("D,group", [(64, 4), (128, 16), (96, 3), (256, 1), (224, 8)])
@pytest.mark.parametrize("power", [20, 30, 36])
def test_queries_of_a_wide_range(mx, power, D, group, room):  # noqa: F811
    """The query's blocks are far apart and the keys' the other way round: every
    block weighs the same in a score.  A query's value may be off by 2^-40 of its
    head's largest where it is under 2^-32 of it."""
    S, n = 16, 300
    c = filled(mx, 20, S, 2, D, False, 6)
    q = rand((1, 2 * group, D), 5).float()
    for i in range(D // 32):
        e = -power if i % 2 else 0
        q[..., 32 * i:32 * i + 32] *= 2.0 ** e
        c.k_scales[..., i] += -power - e + 10
    q, scale = q.to(BF16), 0.02 * 2.0 ** (power - 10)
    table = tables(1, -(-n // S), 20, 1)
    o, lse, _ = mx.cache_attention(q, c, with_room(table, S) if room else table,
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), scale)
    k, v = contents(c, table[0].long(), n)
    for h in range(2):
        qh = q[0, h * group:(h + 1) * group].double()
        top = qh.abs().amax(-1, keepdim=True)
        off = torch.where(qh.abs() < 2.0 ** -32 * top, 2.0 ** -40 * top, 0.0)
        a = scale * (qh @ k[h].T)
        d = scale * ((D + 8) * 2.0 ** -23 * (qh.abs() @ k[h].abs().T) + off @ k[h].abs().T)
        p = torch.softmax(a, -1)
        want = p @ v[h]
        # a weight moves by exp of twice the scores' largest error
        rel = 2.0 ** -10 + torch.expm1(2 * d.amax(-1, keepdim=True)) + n * 2.0 ** -22 + 2.0 ** -19
        bound = rel * (p @ v[h].abs()) + 2.0 ** -23 * v.abs().amax()
        bound += R.unit(BF16) * (want.abs() + bound)
        R.close(o[0, h * group:(h + 1) * group], want, bound)
        R.close(lse[0, h * group:(h + 1) * group], torch.logsumexp(a, -1), d.amax(-1) + n * 2.0 ** -22 + 2.0 ** -17)


@pytest.mark.parametrize("end,window", [(0, 100), (0, 1), (17, 33), (1, 4000)])
@pytest.mark.parametrize("nvfp4", [False, True])
def test_positions_up_to_the_largest_length(mx, end, window, nvfp4):  # noqa: F811
    """The last positions of a length of 2^31 - 2: what lies a few steps past them is
    past 32 signed bits.  The table's pages are all one."""
    S, D = 1549411, 32
    pages = (2 ** 31 - 1) // S                        # S * pages == 2^31 - 2
    n = S * pages - end
    assert S * pages == 2 ** 31 - 2
    c = filled(mx, 1, S, 1, D, nvfp4, 6)
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    q = rand((1, 4, D), 5)
    o, lse, st = mx.cache_attention(q, c, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 0.2,
                                    window=window)
    assert int(st.item()) == 0
    last = (n - 1) % S + 1
    c = c._replace(**{f: getattr(c, f)[:, :, last - window:last] for f in
                      ("k_codes", "k_scales", "v_codes", "v_scales")})
    k, v = contents(c, torch.tensor([0], device="cuda"), window)
    want, bound, wl, bl = R.attention(q[0], k[0], v[0], 0.2, BF16)
    R.close(o[0], want, bound)
    R.close(lse[0], wl, bl)


def test_workspace_is_for_the_device(mx):  # noqa: F811
    """As many warps share the steps as the device's SMs hold (head_dim 64: 4 CTAs of 4
    warps each), whatever GPU it is: parts of 8 heads of 64 with a maximum and a sum, an
    entry of 16 bytes per unit and a word per warp."""
    units, warps = 8, 16 * torch.cuda.get_device_properties(0).multi_processor_count
    want = (units + warps) * 8 * (64 + 2) * 4 + units * 16 + warps * 4
    assert mx.mxfp4_cache_attention_workspace_bytes(1, 8, units, 64, 16, 8192) == want


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("power", [40, 100, 118, -120])
@pytest.mark.parametrize("group", [4, 16])
def test_a_head_of_any_size_leaves_the_others(mx, power, group, room):  # noqa: F811
    """Heads of one kv head whose queries are 2^power times the others'."""
    c = filled(mx, 20, 16, 1, 64, False, 6)
    key_scales(c, 127 + 3, 127 + 6, 3)
    table, n = tables(1, 19, 20, 1), torch.tensor([300], dtype=torch.int32, device="cuda")
    table = with_room(table, 16) if room else table
    q = rand((1, group, 64), 5)
    mixed = q.clone()
    mixed[:, 1::2] = (mixed[:, 1::2].float() * 2.0 ** power).to(BF16)
    o, lse, _ = mx.cache_attention(mixed, c, table, n, 0.01)
    k, v = contents(c, table[0].long()[:19], 300)
    full, bound, fl, bl = R.attention(q[0], k[0], v[0], 0.01, BF16)
    R.close(o[0, ::2], full[::2], bound[::2])
    R.close(lse[0, ::2], fl[::2], bl[::2])


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("gap", [6, 14, 22])
def test_values_of_a_wide_range(mx, gap, room):  # noqa: F811
    """Positions whose weight is 2^gap times the others' hold values 2^-gap times
    theirs: both are half of the output.  Bound: two roundings to 11 bits, and
    products no finer than 2^-37 of the largest weight and scale of a block."""
    S, D, n = 16, 64, 320
    c = make_cache(mx, n // S, S, 1, D, False)
    k, v = torch.zeros((n, 1, D), dtype=BF16, device="cuda"), rand((n, 1, D), 8)
    k[::2, 0, 0] = 4.0
    v[::2] *= 2.0 ** -gap
    mx.cache_write(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), c)
    table = torch.arange(n // S, dtype=torch.int32, device="cuda").view(1, -1)
    q = torch.zeros((1, 2, D), dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    scale = gap * math.log(2.0) / 4.0
    o, _, _ = mx.cache_attention(q, c, with_room(table, S) if room else table,
                                 torch.tensor([n], dtype=torch.int32, device="cuda"), scale)
    kd, vd = contents(c, table[0].long(), n)
    p = torch.softmax(scale * (q[0].double() @ kd[0].T), -1)
    want = p @ vd[0]
    off = (2.0 ** -10 + 2.0 ** -18) * (p @ vd[0].abs()) + n * 2.0 ** -37 * p.amax() * vd.abs().amax()
    R.close(o[0], want, off + R.unit(BF16) * (want.abs() + off) + R.smallest(BF16))

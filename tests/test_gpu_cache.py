"""The paged 4-bit cache: mxfp4_cache_write and mxfp4_cache_read (MXFP4 and
NVFP4, BF16 and FP16) bit for bit against the dense quantizers and the CPU
oracle; mxfp4_cache_attention against a plain 64-bit form; odd sizes, masks,
strides, bad slots, pages and lengths, and what the calls refuse."""
import math

import numpy as np
import pytest
import torch

import decode_reference as R
import oracle
import workloads as W

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import mxfp4_block_quantization_gb300 as m
    return m


def rand(shape, seed, dtype=BF16, std=1.0):
    return W.normal_bf16(shape, seed, std=std, device="cuda").to(dtype)


def make_cache(mx, pages, S, H, D, nvfp4, fill=None):
    g = (torch.tensor([400.0], device="cuda"), torch.tensor([333.0], device="cuda")) if nvfp4 else ()
    c = mx.cache_alloc(pages, S, H, D, *g)
    if fill is not None:
        for t in c[:4]:
            t.fill_(fill)
    return c


def flat_quantized(mx, x, nvfp4, g):
    """codes and flat scales of rows x [n, D], by the dense quantizer."""
    n, D = x.shape
    codes, scales = mx.quantize_nvfp4(x, g) if nvfp4 else mx.quantize(x)
    return codes, R.untile(scales, n, D // (16 if nvfp4 else 32))


def place(slots, S):
    return slots.long() // S, slots.long() % S


CACHES = [(1, 1, 32, 1, 1), (7, 3, 64, 5, 4), (33, 8, 128, 16, 5), (100, 5, 96, 17, 9),
          (257, 2, 256, 64, 6), (64, 1, 160, 3, 40), (300, 4, 192, 100, 4), (3, 130, 32, 2, 3)]


@pytest.mark.parametrize("T,H,D,S,pages", CACHES)
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_write_and_read(mx, T, H, D, S, pages, nvfp4, dtype):
    c = make_cache(mx, pages, S, H, D, nvfp4, fill=0xA5)
    total = pages * S
    T = min(T, total)
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    slots = torch.randperm(total, device="cuda", generator=gen)[:T].to(torch.int32)
    slots[::5] = -1 if T > 1 else slots[::5]
    fused = rand((T, 2 * H + 3, D), T + H, dtype, std=1.7)
    k, v = fused[:, 1:H + 1], fused[:, H + 2:2 * H + 2]
    st = mx.cache_write(k, v, slots, c)
    assert int(st.item()) == 0
    live = slots >= 0
    page, at = place(slots[live], S)
    touched = torch.zeros(pages, S, dtype=torch.bool, device="cuda")
    touched[page, at] = True
    for x, codes, scales, g in ((k, c.k_codes, c.k_scales, c.k_global),
                                (v, c.v_codes, c.v_scales, c.v_global)):
        want_c, want_s = flat_quantized(mx, x[live].reshape(-1, D), nvfp4, g)
        n = int(live.sum())
        assert torch.equal(codes[page, :, at], want_c.view(n, H, -1))
        assert torch.equal(scales[page, :, at], want_s.view(n, H, -1))
        for t in (codes, scales):                    # nothing else was written
            assert (t.transpose(1, 2)[~touched] == 0xA5).all()
    k2, v2, st = mx.cache_read(c, slots, dtype=dtype)
    assert int(st.item()) == 0
    for x, got, codes, scales, g in ((k, k2, c.k_codes, c.k_scales, c.k_global),
                                     (v, v2, c.v_codes, c.v_scales, c.v_global)):
        assert (got[~live] == 0).all()
        if dtype == BF16 and live.any():             # the dense dequantizer's bits
            rows = x[live].reshape(-1, D)
            if nvfp4:
                q, s = mx.quantize_nvfp4(rows, g)
                want = mx.dequantize_nvfp4(q, s, g, rows.shape[0], D)
            else:
                q, s = mx.quantize(rows)
                want = mx.dequantize(q, s, rows.shape[0], D)
            assert torch.equal(got[live].view(torch.int16), want.view(-1, H, D).view(torch.int16))
        want = R.rows_of(codes[page, :, at], scales[page, :, at], nvfp4, 1.0 if g is None else g)
        bound = (R.unit(dtype) + (2.0 ** -21 if nvfp4 else 0.0)) * want.abs() + R.smallest(dtype)
        R.close(got[live], want, bound)


def test_write_against_the_oracle(mx):
    T, H, D, S = 50, 3, 96, 16
    c = make_cache(mx, 4, S, H, D, False)
    k, v = rand((T, H, D), 1), rand((T, H, D), 2, std=1e-3)
    v[3] = 0
    v[4] = (rand((H, D), 3).float() * 2.0 ** -130).to(BF16)
    slots = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")
    mx.cache_write(k, v, slots, c)
    page, at = place(slots, S)
    for x, codes, scales in ((k, c.k_codes, c.k_scales), (v, c.v_codes, c.v_scales)):
        oc, os_ = oracle.quantize(W.bf16_bits(x.reshape(-1, D)))
        flat = R.untile(torch.from_numpy(np.ascontiguousarray(os_)), T * H, D // 32)
        assert np.array_equal(codes[page, :, at].reshape(-1, D // 2).cpu().numpy(), oc)
        assert torch.equal(scales[page, :, at].reshape(-1, D // 32).cpu(), flat)


def test_slots_out_of_range(mx):
    c = make_cache(mx, 3, 4, 2, 64, False, fill=0x11)
    k, v = rand((5, 2, 64), 1), rand((5, 2, 64), 2)
    slots = torch.tensor([0, 12, -2, 11, -1], dtype=torch.int32, device="cuda")
    assert int(mx.cache_write(k, v, slots, c).item()) == mx.MXFP4_EINDEX
    kept = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    kept[0, 0] = kept[2, 3] = False
    assert (c.k_codes.transpose(1, 2)[kept] == 0x11).all()
    assert not (c.k_codes.transpose(1, 2)[~kept] == 0x11).all()
    k2, v2, st = mx.cache_read(c, slots)
    assert int(st.item()) == mx.MXFP4_EINDEX
    assert (k2[[1, 2, 4]] == 0).all() and (v2[[1, 2, 4]] == 0).all() and (k2[0] != 0).any()
    st = mx.cache_write(k[:0], v[:0], slots[:0], c)
    assert int(st.item()) == 0
    assert int(mx.cache_read(c, slots[:0])[2].item()) == 0


def test_read_special_scales(mx):
    for nvfp4, nan in ((False, 255), (True, 0x7F)):
        for dtype in (BF16, F16):
            c = make_cache(mx, 1, 2, 1, 64, nvfp4, fill=0x32)
            c.k_scales.fill_(120)
            c.v_scales.fill_(120)
            c.k_scales[0, 0, 1, 1] = nan
            k, v, _ = mx.cache_read(c, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                    dtype=dtype)
            n = 16 if nvfp4 else 32
            assert torch.isnan(k[1, 0, n:2 * n]).all() and not torch.isnan(k[1, 0, :n]).any()
            assert not torch.isnan(k[0]).any() and not torch.isnan(v).any()


def test_cache_past_32_bits(mx):
    """A cache of more than 2^32 bytes of codes: write, read and attention at its end."""
    H, S, D = 8, 64, 256
    pages = 2 ** 32 // (H * S * D // 2) + 4
    c = make_cache(mx, pages, S, H, D, False)
    T = 70
    k, v = rand((T, H, D), 1), rand((T, H, D), 2)
    first = (pages - 2) * S
    slots = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
    assert int(mx.cache_write(k, v, slots, c).item()) == 0
    want_c, _ = flat_quantized(mx, k.reshape(-1, D), False, None)
    page, at = place(slots, S)
    assert torch.equal(c.k_codes[page, :, at].reshape(-1, D // 2), want_c)
    k2, v2, _ = mx.cache_read(c, slots)
    assert torch.equal(k2, mx.dequantize(*mx.quantize(k.reshape(-1, D)), T * H, D).view(T, H, D))
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    check_attention(mx, rand((1, H * 2, D), 3), c, table, lens, 0.06)


# ------------------------------------------------------------- attention
def check_attention(mx, q, c, table, lens, scale, window=0, status=0):
    B, Hq, D = q.shape
    H = c.k_codes.shape[1]
    nvfp4 = c.k_global is not None
    out = torch.full((B, Hq, D), 99.0, dtype=q.dtype, device="cuda")
    o, lse, st = mx.cache_attention(q, c, table, lens, scale, window=window, out=out)
    assert int(st.item()) == status
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        S = c.k_codes.shape[2]
        pages = table[b].long()[:-(-n // S)]

        def rows(codes, scales, g):
            x = R.rows_of(codes[pages], scales[pages], nvfp4, 1.0 if g is None else g)
            return x.transpose(0, 1).flatten(1, 2)[:, lo:n]          # [H, positions, D]

        k, v = rows(c.k_codes, c.k_scales, c.k_global), rows(c.v_codes, c.v_scales, c.v_global)
        G = Hq // H
        for h in range(H):
            want, bound, wl, bl = R.attention(q[b, h * G:(h + 1) * G], k[h], v[h], scale, q.dtype)
            R.close(o[b, h * G:(h + 1) * G], want, bound)
            R.close(lse[b, h * G:(h + 1) * G], wl, bl)
    return o, lse


def filled(mx, pages, S, H, D, nvfp4, seed, dtype=BF16):
    c = make_cache(mx, pages, S, H, D, nvfp4)
    n = pages * S
    mx.cache_write(rand((n, H, D), seed, dtype), rand((n, H, D), seed + 1, dtype),
                   torch.arange(n, dtype=torch.int32, device="cuda"), c)
    return c


def tables(B, per, pages, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.stack([torch.randperm(pages, device="cuda", generator=gen)[:per]
                        for _ in range(B)]).to(torch.int32)


SHAPES = [  # lens, q heads, kv heads, D, page size
    ([1], 1, 1, 32, 1), ([5, 1, 0, 16, 17], 8, 2, 64, 16), ([63, 64, 65, 128, 3], 32, 4, 128, 64),
    ([700], 64, 8, 128, 16), ([31, 200, 33], 6, 2, 96, 7), ([129, 77], 16, 1, 256, 32),
    ([100, 90], 40, 5, 160, 10), ([500, 3], 24, 1, 192, 100), ([1000, 999], 12, 12, 64, 24),
    ([20, 45], 20, 1, 224, 5), ([3000, 2049, 1], 7, 1, 128, 48), ([12000], 8, 1, 64, 128)]


@pytest.mark.parametrize("lens,Hq,H,D,S", SHAPES)
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention(mx, lens, Hq, H, D, S, nvfp4, dtype):
    B, per = len(lens), -(-max(lens) // S) + 1
    c = filled(mx, per * 2 + 1, S, H, D, nvfp4, D + S, dtype)
    table = tables(B, per, per * 2 + 1, 3)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = rand((B, Hq, D), 5, dtype)
    check_attention(mx, q, c, table, n, D ** -0.5)
    check_attention(mx, q, c, table, n, 1.1, window=40)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 64, 1000, 5000])
def test_attention_windows(mx, window):
    c = filled(mx, 70, 16, 2, 64, False, 9)
    n = torch.tensor([1000, 16, 65, 0, 1], dtype=torch.int32, device="cuda")
    check_attention(mx, rand((5, 8, 64), 4), c, tables(5, 64, 70, 1), n, 0.3, window=window)


def test_attention_many_sequences(mx):
    rng = np.random.default_rng(3)
    lens = torch.from_numpy(rng.integers(0, 400, 200).astype(np.int32)).cuda()
    c = filled(mx, 60, 32, 2, 64, True, 2)
    check_attention(mx, rand((200, 10, 64), 1), c, tables(200, 13, 60, 5), lens, 0.125)


def test_attention_strided_query_and_table(mx):
    c = filled(mx, 20, 16, 2, 64, False, 9)
    fused = rand((3, 12, 96), 7)
    table = tables(3, 10, 20, 2)
    wide = torch.full((3, 17), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :10] = table
    n = torch.tensor([130, 7, 160], dtype=torch.int32, device="cuda")
    check_attention(mx, fused[:, 2:10, 16:80], c, wide[:, :10], n, 0.2)


def test_attention_bytes_outside_the_range_never_matter(mx):
    """Codes and scales of every position that is masked hold NaN scales; the
    table's entries past a length hold wild pages."""
    S, H, D = 16, 2, 128
    for nvfp4, nan in ((False, 255), (True, 0x7F)):
        c = filled(mx, 12, S, H, D, nvfp4, 1)
        n = torch.tensor([37, 5, 0], dtype=torch.int32, device="cuda")
        table = torch.tensor([[3, 7, 1, -5], [9, 10 ** 9, -1, 4], [-1, -1, -1, -1]],
                             dtype=torch.int32, device="cuda")
        live = torch.zeros(12, S, dtype=torch.bool, device="cuda")
        live[3], live[7], live[1, :5], live[9, :5] = True, True, True, True
        for t in (c.k_scales, c.v_scales):
            t.transpose(1, 2)[~live] = nan
        check_attention(mx, rand((3, 16, D), 2), c, table, n, 0.1)
        live[3], live[7, :3], live[9, :3] = False, False, False
        for t in (c.k_scales, c.v_scales):
            t.transpose(1, 2)[~live] = nan
        n[1] = 5
        o, _, _ = mx.cache_attention(rand((3, 16, D), 2), c, table, n, 0.1, window=2)
        assert torch.isfinite(o).all()


def test_attention_nan_in_range_stays_in_its_head(mx):
    c = filled(mx, 4, 16, 2, 64, False, 1)
    n = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1, 2], [3, 3, 3]], dtype=torch.int32, device="cuda")
    c.k_scales[1, 1, 4, 0] = 255
    o, lse, _ = mx.cache_attention(rand((2, 8, 64), 3), c, table, n, 0.1)
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all()


def test_attention_status(mx):
    c = filled(mx, 6, 16, 1, 64, False, 4)
    table = torch.tensor([[0, 1], [2, 77], [4, -3], [5, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([32, 20, 16, 33], dtype=torch.int32, device="cuda")
    q = rand((4, 4, 64), 5)
    o, lse, st = mx.cache_attention(q, c, table, n, 0.2)
    assert int(st.item()) == mx.MXFP4_EINDEX
    assert (o[3] == 0).all() and (lse[3] == -math.inf).all()          # length past the table
    short = n.clone()
    short[1], short[3] = 16, 0                                        # the positions that remain
    want = check_attention(mx, q, c, table.clamp(0, 5), short, 0.2)
    bound = 2.0 ** -7 * want[0].double().abs() + 2.0 ** -9
    R.close(o, want[0], bound)
    n[3] = -1
    assert int(mx.cache_attention(q, c, table, n, 0.2)[2].item()) == mx.MXFP4_EINDEX
    n[3], n[1] = 0, 16
    assert int(mx.cache_attention(q, c, table, n, 0.2)[2].item()) == mx.MXFP4_OK


def test_attention_large_scores(mx):
    """Scores far apart and far from zero: the running maximum keeps the sums finite."""
    c = filled(mx, 20, 16, 1, 64, False, 4)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    for scale in (30.0, -30.0, 0.0):
        check_attention(mx, rand((1, 4, 64), 5) * 3, c, tables(1, 19, 20, 1), n, scale)


def test_attention_scales_of_every_size(mx):
    """Keys and values of very large and very small magnitude."""
    for power in (-60, -20, 20, 60):
        c = make_cache(mx, 10, 16, 2, 64, False)
        k = (rand((160, 2, 64), 1).float() * 2.0 ** power).to(BF16)
        v = (rand((160, 2, 64), 2).float() * 2.0 ** -power).to(BF16)
        mx.cache_write(k, v, torch.arange(160, dtype=torch.int32, device="cuda"), c)
        n = torch.tensor([150], dtype=torch.int32, device="cuda")
        check_attention(mx, rand((1, 8, 64), 5), c, tables(1, 10, 10, 1), n, 0.125 * 2.0 ** -power)


def test_attention_same_bits_on_every_call_and_stream(mx):
    c = filled(mx, 300, 16, 2, 128, False, 4)
    q, table = rand((2, 16, 128), 5), tables(2, 256, 300, 1)
    n = torch.tensor([4096, 3001], dtype=torch.int32, device="cuda")
    o, lse, _ = mx.cache_attention(q, c, table, n, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [mx.cache_attention(q, c, table, n, 0.1, stream=s) for _ in range(4)]
    s.synchronize()
    for a, b, _ in got:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_decode_in_a_graph(mx):
    """Write, attention and read of a growing sequence, replayed from one graph."""
    H, D, S = 2, 64, 16
    c = filled(mx, 8, S, H, D, True, 4)
    table = tables(1, 8, 8, 1)
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = rand((1, 8, D), 1), rand((1, H, D), 2), rand((1, H, D), 3)

    def step():
        st = mx.cache_write(k, v, slots, c)
        return mx.cache_attention(q, c, table, n, 0.1)[:2] + mx.cache_read(c, slots)[:2] + (st,)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse, k2, v2, st = step()
    for i in range(60, 70):
        slots.fill_(int(table[0, i // S]) * S + i % S)
        n.fill_(i + 1)
        for t, seed in ((q, i), (k, 100 + i), (v, 200 + i)):
            t.copy_(rand(tuple(t.shape), seed))
        g.replay()
        want, wl = check_attention(mx, q, c, table, n, 0.1)
        assert torch.equal(o, want) and torch.equal(lse, wl) and int(st.item()) == 0
        q2, s2 = mx.quantize_nvfp4(k.view(H, D), c.k_global)
        assert torch.equal(k2[0], mx.dequantize_nvfp4(q2, s2, c.k_global, H, D))


def test_refusals(mx):
    c = make_cache(mx, 4, 16, 2, 64, False, fill=7)
    k = rand((3, 2, 64), 1)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    n = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    q = rand((3, 4, 64), 2)
    odd = rand((3, 2, 68), 1)[:, :, :64]
    bad = [lambda: mx.cache_write(k.float(), k.float(), slots, c),
           lambda: mx.cache_write(k, k.to(F16), slots, c),
           lambda: mx.cache_write(k[:2], k, slots, c),
           lambda: mx.cache_write(k, k, slots.long(), c),
           lambda: mx.cache_write(k, k, slots, c._replace(k_scales=c.k_scales[..., :1])),
           lambda: mx.cache_write(k, k, slots, c._replace(k_global=torch.ones(1, device="cuda"))),
           lambda: mx.cache_write(k.transpose(1, 2), k, slots, c),
           lambda: mx.cache_read(c, slots, k_out=k[:2].clone(), v_out=k.clone()),
           lambda: mx.cache_read(c, slots, dtype=torch.float32),
           lambda: mx.cache_attention(q[:, :, :32], c, table, n, 1.0),
           lambda: mx.cache_attention(q, c, table[:2], n, 1.0),
           lambda: mx.cache_attention(q, c, table, n[:2], 1.0),
           lambda: mx.cache_attention(q, c, table, n, 1.0, out=q.to(F16)),
           lambda: mx.cache_attention(q.cpu(), c, table, n, 1.0)]
    for fn in bad:
        with pytest.raises(ValueError):
            fn()
    codes = [lambda: mx.cache_write(odd, odd, slots, c),                       # strides % 8
             lambda: mx.cache_attention(q[:, :3], c, table, n, 1.0),          # 3 heads over 2
             lambda: mx.cache_attention(q, c, table, n, math.inf),
             lambda: mx.cache_attention(q, c, table, n, 1.0, window=-1),
             lambda: mx.cache_read(c, slots, k_out=c.k_codes.view(BF16).view(-1)[:384], v_out=k.clone())]
    for fn in codes:
        with pytest.raises(mx.MXFP4Error):
            fn()
    torch.cuda.synchronize()
    for t in c[:4]:
        assert (t == 7).all()
    wide = mx.cache_alloc(1, 4, 1, 288)                                       # head_dim > 256
    with pytest.raises(mx.MXFP4Error):
        mx.cache_attention(rand((1, 1, 288), 1), wide, table[:1, :1], n[:1], 1.0)

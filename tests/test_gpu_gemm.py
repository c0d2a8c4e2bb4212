"""Products of 4-bit activations with 4-bit weights, dense and per expert,
against the 64-bit form within bounds derived from the sums' lengths."""
import pytest
import torch

import decode_reference as R
import layer_reference as L

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operand(rows, K, nv, g, pad=255):
    """Random codes and tiled scales [rows, K]; the bytes that pad the scales
    hold `pad` (255: NaN in E8M0; 127 in E4M3)."""
    per = 16 if nv else 32
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    flat = torch.full((-(-rows // 128) * 128, -(-K // (4 * per)) * 4), 127 if nv and pad == 255 else pad,
                      dtype=torch.uint8, device="cuda")
    lo, hi = (40, 72) if nv else (121, 130)
    flat[:rows, :K // per] = torch.randint(lo, hi, (rows, K // per), dtype=torch.uint8, device="cuda", generator=g)
    mt, kt = flat.shape[0] // 128, flat.shape[1] // 4
    return codes, flat.view(mt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def half(g, dtype, *shape, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def dense(mx, T, N, K, nv=False, dtype=BF, bias=False, act=None, gate=None, residual=False, seed=0, pad=255):
    g = gen(seed + 7 * T + 3 * N + K)
    xc, xs = operand(T, K, nv, g, pad)
    wc, ws = operand(N, K, nv, g, pad)
    xg, wg = (torch.tensor([v], device="cuda") for v in (3.5, 0.75 * max(K, 1) ** 0.5))
    cols = N // 2 if gate else N
    b = half(g, dtype, N) if bias else None
    r = half(g, dtype, T, cols) if residual else None
    kw = dict(bias=b, activation=act, gate=gate, residual=r, out_dtype=dtype)
    y = mx.gemm_nvfp4(xc, xs, xg, wc, ws, wg, **kw) if nv else mx.gemm(xc, xs, wc, ws, **kw)
    x, w = (R.weights(c, s, nv, v) if K else torch.zeros(c.shape[0], 0, dtype=torch.float64, device="cuda")
            for c, s, v in ((xc, xs, xg), (wc, ws, wg)))
    assert y.dtype is dtype
    L.close(y, *L.gemm(x, w, dtype, b, act, gate, r))
    return y


# tokens around the tiles' edges, weights around theirs, K's steps of 64 and
# stages of 256, and what is left of them
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 96)])
def test_tokens(mx, T, N, K):
    dense(mx, T, N, K)
    dense(mx, T, N, K, nv=True, dtype=FP)


@pytest.mark.parametrize("N", [1, 2, 31, 64, 127, 129, 255, 257, 384, 1000])
@pytest.mark.parametrize("T", [3, 130])
def test_weight_rows(mx, T, N):
    dense(mx, T, N, 160, bias=True, residual=True)
    dense(mx, T, N, 288, nv=True, bias=True)


@pytest.mark.parametrize("K", [0, 32, 64, 96, 128, 192, 224, 256, 288, 512, 544, 768, 1024, 1312, 2048, 2880, 7168])
@pytest.mark.parametrize("nv", [False, True])
def test_sums_lengths(mx, K, nv):
    dense(mx, 5, 130, K, nv=nv, bias=True)
    dense(mx, 140, 130, K, nv=nv, dtype=FP, residual=True)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gate", [None, "first", "second"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_epilogue(mx, act, gate, dtype):
    for T in (4, 150):
        dense(mx, T, 264, 128, dtype=dtype, bias=True, act=act, gate=gate, residual=True)
        dense(mx, T, 512, 320, nv=True, dtype=dtype, act=act, gate=gate)


@pytest.mark.parametrize("N", [2, 6, 62, 64, 130, 192, 254, 256, 258, 320, 510, 514, 770, 1152])
@pytest.mark.parametrize("nv", [False, True])
def test_halves_of_any_size(mx, N, nv):
    """The second half's scales begin anywhere in a tile of 128 rows."""
    for T in (3, 129):
        dense(mx, T, N, 192, nv=nv, bias=True, act="silu", gate="first")
        dense(mx, T, N, 320, nv=nv, gate="second", act="gelu")


@pytest.mark.parametrize("T,N,K", [(1, 7168, 2048), (24, 4096, 1536), (300, 3000, 1024), (1024, 2048, 768), (2, 19500, 512)])
@pytest.mark.parametrize("nv", [False, True])
def test_larger(mx, T, N, K, nv):
    dense(mx, T, N, K, nv=nv, bias=True, residual=True)
    dense(mx, T, N, K, nv=nv, act="silu", gate="second")


@pytest.mark.parametrize("nv", [False, True])
def test_equal_calls_give_equal_bits(mx, nv):
    for T, N, K in ((1, 1024, 7168), (16, 2048, 4096), (700, 1500, 1024)):
        assert torch.equal(dense(mx, T, N, K, nv=nv).view(torch.int16), dense(mx, T, N, K, nv=nv).view(torch.int16))


@pytest.mark.parametrize("T", [5, 140])
def test_scales_of_any_exponent(mx, T):
    """2^-60 to 2^60 in one sum: the bound is each sum's own magnitudes."""
    g = gen(9)
    K, N = 256, 140
    (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
    for s, n in ((xs, T), (ws, N)):
        s[s < 200] = torch.randint(67, 188, (int((s < 200).sum()),), dtype=torch.uint8, device="cuda", generator=g)
    y = mx.gemm(xc, xs, wc, ws)
    L.close(y, *L.gemm(R.weights(xc, xs, False), R.weights(wc, ws, False), BF))


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("T", [5, 140])
def test_a_scale_of_nan_stays_in_its_row(mx, nv, T):
    g = gen(10)
    K, N = 192, 150
    (xc, xs), (wc, ws) = operand(T, K, nv, g), operand(N, K, nv, g)
    nan = 127 if nv else 255
    xs[(3 % 32) * 16] = nan                       # row 3, first block
    ws[512 * -(-K // (64 if nv else 128)) + 5 * 16 + 1] = nan   # row 133, second block
    one = torch.ones(1, device="cuda")
    y = mx.gemm_nvfp4(xc, xs, one, wc, ws, one) if nv else mx.gemm(xc, xs, wc, ws)
    want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    want[3], want[:, 133] = True, True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("T", [5, 140])
def test_global_scales_far_apart(mx, T):
    """Global scales whose product, or its inverse, no float32 holds: sums of zero
    stay zero, and the others are what two divisions make of them."""
    g = gen(15)
    K, N = 128, 40
    (xc, xs), (wc, ws) = operand(T, K, True, g), operand(N, K, True, g)
    xc[1], wc[3] = 0, 0
    for a, b in ((2.0 ** -100, 2.0 ** -100), (2.0 ** 100, 2.0 ** -100), (2.0 ** 70, 2.0 ** 80)):
        ga, gb = torch.tensor([a], device="cuda"), torch.tensor([b], device="cuda")
        y = mx.gemm_nvfp4(xc, xs, ga, wc, ws, gb)
        want, bound = L.gemm(R.weights(xc, xs, True), R.weights(wc, ws, True), BF)
        L.close(y, want / a / b, bound / a / b + R.smallest(BF) + 2.0 ** -126)
        assert (y[1] == 0).all() and (y[:, 3] == 0).all()


def test_strides_and_places(mx):
    """y and the residual at odd addresses with odd strides, and the residual in y."""
    g = gen(11)
    T, N, K = 37, 70, 96
    (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
    x, w = R.weights(xc, xs, False), R.weights(wc, ws, False)
    buffer = half(g, BF, T * 75 + 9)
    before = buffer.clone()
    y = buffer[3:3 + T * 75].view(T, 75)[:, 1:71]
    residual = half(g, BF, T, 101)[:, 20:90]
    mx.mxfp4_gemm(xc, xs, wc, ws, y, residual=residual)
    L.close(y, *L.gemm(x, w, BF, residual=residual))
    apart = torch.ones_like(buffer, dtype=torch.bool)
    apart[3:3 + T * 75].view(T, 75)[:, 1:71] = False
    assert torch.equal(buffer[apart], before[apart])
    old = half(g, BF, T, N)
    y = old.clone()
    mx.mxfp4_gemm(xc, xs, wc, ws, y, residual=y)
    L.close(y, *L.gemm(x, w, BF, residual=old))


def test_rows_behind_the_sizes_are_left(mx):
    g = gen(12)
    for T, N, K in ((3, 50, 64), (130, 129, 64), (257, 300, 32)):
        (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
        big = torch.full((T + 300, N), 7.0, dtype=BF, device="cuda")
        mx.mxfp4_gemm(xc, xs, wc, ws, big[:T])
        assert (big[T:] == 7).all()


# ----------------------------------------------------------------- per expert
def batch(sizes, K, nv, g, extra=0):
    """Rows of a routed batch by expert: codes, scales as the grouped calls
    write them (255 or 127 in every byte that pads), and the rows' values."""
    rows = sum(sizes) + extra
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    parts, values, at = [], [], 0
    gs = (torch.rand(len(sizes), device="cuda", generator=g) + 0.5) * 4
    for e, n in enumerate(sizes):
        _, s = operand(n, K, nv, g)
        parts.append(s)
        if n:
            values.append(R.weights(codes[at:at + n], s, nv, gs[e]))
        at += n
    per = 16 if nv else 32
    bound = (rows + 127 * len(sizes)) // 128 * 128 * (-(-K // (4 * per)) * 4)
    scales = torch.full((max(bound, 16),), 127 if nv else 255, dtype=torch.uint8, device="cuda")
    flat = torch.cat(parts) if parts else scales[:0]
    scales[:flat.numel()] = flat
    off = torch.tensor([0] + list(sizes), device="cuda").cumsum(0).to(torch.int32)
    return codes, scales, off, values, gs


def experts(mx, sizes, N, K, nv=False, dtype=BF, bias=False, act=None, gate=None, seed=0, extra=0):
    g = gen(seed + N + K + len(sizes))
    E = len(sizes)
    xc, xs, off, values, xg = batch(sizes, K, nv, g, extra)
    w = [operand(N, K, nv, g) for _ in range(E)]
    wc, ws = torch.stack([c for c, _ in w]), torch.cat([s for _, s in w])
    wg = (torch.rand(E, device="cuda", generator=g) + 0.5) * 2
    b = half(g, dtype, E, N) if bias else None
    cols = N // 2 if gate else N
    y = torch.full((sum(sizes) + extra, cols), 7.0, dtype=dtype, device="cuda")
    kw = dict(bias=b, activation=act, gate=gate, out=y)
    if nv:
        y, status = mx.moe_gemm_nvfp4(xc, xs, xg, off, wc, ws, wg, **kw)
    else:
        y, status = mx.moe_gemm(xc, xs, off, wc, ws, **kw)
    assert int(status) == 0
    at, i = 0, 0
    for e, n in enumerate(sizes):
        if n:
            L.close(y[at:at + n], *L.gemm(values[i], R.weights(wc[e], w[e][1], nv, wg[e]), dtype,
                                          None if b is None else b[e], act, gate))
            i += 1
        at += n
    assert (y[at:] == 7).all()
    return y


@pytest.mark.parametrize("sizes", [[5], [0, 0, 3], [1, 0, 2, 127, 128, 129, 0], [256, 255, 257, 1], [0] * 40 + [700],
                                   [2] * 70, [130, 0, 0, 0, 1]])
@pytest.mark.parametrize("nv", [False, True])
def test_segments(mx, sizes, nv):
    experts(mx, sizes, 130, 160, nv=nv, bias=True, extra=9)
    experts(mx, sizes, 256, 256, nv=nv, dtype=FP, act="silu", gate="second", extra=140)


@pytest.mark.parametrize("N", [2, 100, 320, 514])
def test_segments_halves(mx, N):
    experts(mx, [3, 140, 0, 20], N, 96, bias=True, act="silu", gate="first")
    experts(mx, [3, 140, 0, 20], N, 96, nv=True, bias=True, act="gelu_tanh", gate="second")


def test_many_experts(mx):
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 3, (1500,), generator=g).tolist()
    sizes[77] = 300
    experts(mx, sizes, 64, 64, bias=True)


def test_no_rows(mx):
    experts(mx, [0, 0, 0], 64, 64, extra=5)
    experts(mx, [0], 64, 64)
    empty = torch.zeros(0, 32, dtype=torch.uint8, device="cuda")
    y, status = mx.moe_gemm(empty, torch.zeros(0, dtype=torch.uint8, device="cuda"),
                            torch.zeros(1, dtype=torch.int32, device="cuda"),
                            torch.zeros(0, 8, 32, dtype=torch.uint8, device="cuda"), empty.view(-1))
    assert y.shape == (0, 8) and int(status) == 0


def test_no_terms_leave_the_bias(mx):
    experts(mx, [2, 0, 150], 70, 0, bias=True)
    experts(mx, [2, 0, 150], 70, 0, bias=True, act="silu", gate="first", nv=True)


@pytest.mark.parametrize("bad", [[1, 5, 9, 12], [0, 6, 5, 12], [0, 5, 9, 13], [0, -1, 9, 12], [0, 5, 2 ** 31 - 1, 12]])
def test_bad_offsets(mx, bad):
    g = gen(13)
    xc, xs, _, _, _ = batch([5, 4, 3], 64, False, g)
    w = [operand(40, 64, False, g) for _ in range(3)]
    y = torch.full((12, 40), 7.0, dtype=BF, device="cuda")
    _, status = mx.moe_gemm(xc, xs, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                            torch.stack([c for c, _ in w]), torch.cat([s for _, s in w]), out=y)
    assert int(status) == mx.MXFP4_EOFFSETS and (y == 7).all()


def test_refusals(mx):
    g = gen(14)
    (xc, xs), (wc, ws) = operand(6, 64, False, g), operand(10, 64, False, g)
    with pytest.raises(ValueError, match="y must"):
        mx.mxfp4_gemm(xc, xs, wc, ws, torch.empty(6, 11, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="bias"):
        mx.gemm(xc, xs, wc, ws, bias=torch.zeros(10, device="cuda"))
    with pytest.raises(ValueError, match="residual"):
        mx.gemm(xc, xs, wc, ws, residual=torch.zeros(5, 10, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="activation"):
        mx.gemm(xc, xs, wc, ws, activation="tanh")
    with pytest.raises(ValueError, match="gate"):
        mx.gemm(xc, xs, wc, ws, gate="both")
    with pytest.raises(ValueError, match="x_scales"):
        mx.gemm(xc, xs[:100], wc, ws)
    with pytest.raises(ValueError, match="elements per row"):
        mx.gemm(xc[:, :16].contiguous(), xs, wc, ws)
    with pytest.raises(ValueError, match="global_scale"):
        mx.gemm_nvfp4(xc, xs, None, wc, ws, None)
    with pytest.raises(ValueError, match="bfloat16 or torch.float16"):
        mx.gemm(xc, xs, wc, ws, out_dtype=torch.float32)
    with pytest.raises(mx.MXFP4Error):                      # 2 x 24 elements: not in pieces of 32
        mx.gemm(xc[:, :24].contiguous(), xs, wc[:, :24].contiguous(), ws)
    y = torch.zeros(12, 10, dtype=BF, device="cuda")
    with pytest.raises(mx.MXFP4Error):
        mx.mxfp4_gemm(xc, xs, wc, ws, y[:6], residual=y[1:7])

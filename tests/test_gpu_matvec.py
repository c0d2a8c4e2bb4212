"""Products with 4-bit weights (mxfp4_matvec, mxfp4_moe_matvec and their
NVFP4 and FP16 forms) against plain 64-bit ones, at the sizes, strides,
scales and routings where they can go wrong, and what they refuse."""
import math

import numpy as np
import pytest
import torch

import decode_reference as R
import workloads as W

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import mxfp4_block_quantization_gb300 as m
    return m


def rand(shape, seed, dtype=BF16, std=1.0):
    return W.normal_bf16(shape, seed, std=std, device="cuda").to(dtype)


def make_weights(mx, N, K, nvfp4, seed):
    w = rand((N, K), seed, std=0.02)
    if nvfp4:
        g = torch.full((1,), 448.0 * 6.0 / 0.11, device="cuda")
        return (*mx.quantize_nvfp4(w, g), g)
    return (*mx.quantize(w), None)


def call(mx, x, codes, scales, g, **kw):
    if g is None:
        return mx.matvec(x, codes, scales, **kw)
    return mx.matvec_nvfp4(x, codes, scales, g, **kw)


def check(mx, x, codes, scales, g, dtype=None):
    dtype = dtype or x.dtype
    T, N = x.shape[0], codes.shape[0]
    buf = torch.full((T, N + 3), 77.0, dtype=dtype, device="cuda")   # guard columns
    y = call(mx, x, codes, scales, g, out=buf[:, :N])
    w = R.weights(codes, scales, g is not None, 1.0 if g is None else g)
    want, bound = R.product(x, w, dtype)
    R.close(y, want, bound)
    assert (buf[:, N:] == 77.0).all(), "wrote past a row of y"
    return y


SIZES = [(1, 1, 32), (1, 16, 64), (2, 5, 96), (3, 127, 160), (7, 129, 128), (8, 300, 2880),
         (9, 33, 512), (16, 1001, 288), (17, 256, 1056), (32, 64, 2048), (33, 130, 736),
         (65, 17, 320), (1, 4097, 768), (5, 2048, 7168), (1, 640, 16384)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_matvec(mx, T, N, K, nvfp4, dtype):
    codes, scales, g = make_weights(mx, N, K, nvfp4, T * 7 + N + K)
    x = rand((T, K), T + N * 3 + K, dtype)
    check(mx, x, codes, scales, g)
    check(mx, x, codes, scales, g, F32)


@pytest.mark.parametrize("T,N,K", [(1, 100, 16), (4, 130, 48), (9, 31, 80), (2, 1000, 2896)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_matvec_nvfp4_odd_blocks(mx, T, N, K, dtype):
    """K a multiple of 16 only: rows of codes start at 8-byte boundaries."""
    codes, scales, g = make_weights(mx, N, K, True, K)
    check(mx, rand((T, K), K + 1, dtype), codes, scales, g, F32)


@pytest.mark.parametrize("nvfp4", [False, True])
def test_matvec_strided_x_and_single_rows(mx, nvfp4):
    codes, scales, g = make_weights(mx, 200, 256, nvfp4, 1)
    wide = rand((6, 320), 2)
    check(mx, wide[:, 64:], codes, scales, g)
    check(mx, wide[::2, :256], codes, scales, g)
    check(mx, wide[3:4, 8:264], codes, scales, g)


def test_matvec_empty(mx):
    codes, scales, _ = make_weights(mx, 40, 64, False, 3)
    assert call(mx, rand((0, 64), 1), codes, scales, None).shape == (0, 40)
    x = torch.empty((3, 0), dtype=BF16, device="cuda")
    y = torch.full((3, 40), 5.0, dtype=BF16, device="cuda")
    empty = torch.empty((40, 0), dtype=torch.uint8, device="cuda")
    call(mx, x, empty, scales, None, out=y)
    assert (y == 0).all(), "an empty sum is zero"


def random_scaled(N, K, lo, hi, seed, nvfp4=False):
    """Random codes and random scale bytes in [lo, hi], in the tiled layout."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    cols = K // (16 if nvfp4 else 32)
    n = -(-N // 128) * 128 * (-(-cols // 4) * 4)
    scales = torch.randint(lo, hi + 1, (n,), device="cuda", generator=gen).to(torch.uint8)
    return codes, scales


@pytest.mark.parametrize("lo,hi,power", [(0, 60, 100), (100, 150, 0), (190, 254, -110),
                                         (0, 254, -20)])
def test_matvec_every_scale(mx, lo, hi, power):
    """Scale bytes over the whole range, 0 (2^-127) among them: the weights
    are 2^(s-127) multiples whatever the neighbours' are."""
    codes, scales = random_scaled(70, 256, lo, hi, lo + hi)
    x = (rand((5, 256), 9).float() * 2.0 ** power).to(BF16)
    y = mx.matvec(x, codes, scales, out_dtype=F32)
    want, bound = R.product(x, R.weights(codes, scales, False), F32)
    big = want.abs() > 3.0e38                       # past float32: infinite in either form
    y, want = torch.where(big, 0.0, y), torch.where(big, 0.0, want)
    mass = x.double().abs() @ R.weights(codes, scales, False).abs().T
    fine = mass < 1.0e38                            # no partial sum overflows
    R.close(torch.where(fine, y, 0.0), torch.where(fine, want, 0.0), bound)
    assert fine.any()


def test_matvec_nvfp4_every_scale(mx):
    codes, scales = random_scaled(130, 320, 0, 126, 4, nvfp4=True)
    for g in (1.0, 3.0e-5, 7.0e6):
        check(mx, rand((3, 320), 8), codes, scales, torch.tensor([g], device="cuda"), F32)


def test_matvec_nan_scales_stay_in_their_rows(mx):
    codes, scales, _ = make_weights(mx, 150, 256, False, 6)
    row, col = 137, 5
    scales[((row // 128) * 2 + col // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + col % 4] = 255
    y = mx.matvec(rand((9, 256), 3), codes, scales)
    assert torch.isnan(y[:, row]).all()
    assert torch.isfinite(torch.cat((y[:, :row], y[:, row + 1:]), 1)).all()
    n_codes, n_scales, g = make_weights(mx, 150, 256, True, 6)
    n_scales[((row // 128) * 4 + col // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + col % 4] = 0x7F
    y = mx.matvec_nvfp4(rand((9, 256), 3), n_codes, n_scales, g)
    assert torch.isnan(y[:, row]).all()
    assert torch.isfinite(torch.cat((y[:, :row], y[:, row + 1:]), 1)).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_matvec_infinite_and_nan_inputs_stay_in_their_rows(mx, dtype):
    codes, scales, _ = make_weights(mx, 70, 128, False, 5)
    codes[:, 3] = 0x22                       # elements 6 and 7 of every row: 1.0
    scales.fill_(127)
    x = rand((10, 128), 6, dtype)
    x[1, 6] = math.inf
    x[4, 7] = -math.inf
    x[7, 6] = math.nan
    y = mx.matvec(x, codes, scales, out_dtype=F32)
    want = x.double() @ R.weights(codes, scales, False).T
    assert (y[1] == math.inf).all() and (y[4] == -math.inf).all() and torch.isnan(y[7]).all()
    rest = [0, 2, 3, 5, 6, 8, 9]
    ref, bound = R.product(x[rest], R.weights(codes, scales, False), F32)
    R.close(y[rest], ref, bound)
    assert torch.equal(torch.isnan(want), torch.isnan(y.double()))


@pytest.mark.parametrize("spread", [20, 60, 120])
def test_matvec_wide_range_of_x(mx, spread):
    """Elements of one row over many binades, subnormals among them."""
    codes, scales, _ = make_weights(mx, 90, 512, False, 7)
    gen = torch.Generator(device="cuda").manual_seed(spread)
    e = torch.rand((6, 512), device="cuda", generator=gen) * 2 * spread - spread
    x = (rand((6, 512), 11).float() * torch.exp2(e)).to(BF16)
    x[2] = (rand((512,), 12).float() * 2.0 ** -128).to(BF16)     # subnormal BF16
    check(mx, x, codes, scales, None, F32)


def test_matvec_same_bits_on_every_call_and_stream(mx):
    codes, scales, _ = make_weights(mx, 1000, 2048, False, 8)
    x = rand((4, 2048), 9)
    want = mx.matvec(x, codes, scales, out_dtype=F32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = [mx.matvec(x, codes, scales, out_dtype=F32, stream=s) for _ in range(4)]
    s.synchronize()
    for y in out:
        assert torch.equal(y, want)


def test_matvec_in_a_graph(mx):
    codes, scales, _ = make_weights(mx, 256, 512, False, 10)
    x = rand((2, 512), 1)
    y = mx.matvec(x, codes, scales)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.matvec(x, codes, scales, out=y)
    x.copy_(rand((2, 512), 2))
    g.replay()
    want, bound = R.product(x, R.weights(codes, scales, False), BF16)
    R.close(y, want, bound)


# ------------------------------------------------------------ experts
def route(mx, T, k, E, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    off, dest, rows, st = mx.moe_route(torch.from_numpy(ids).cuda(), E)
    return off, rows


def make_experts(mx, E, N, K, nvfp4, seed):
    w = rand((E, N, K), seed, std=0.02)
    g = (448.0 * 6.0 / 0.11 * (1.0 + torch.arange(E, device="cuda") / E)).float() if nvfp4 else None
    q = [mx.quantize_nvfp4(w[e], g[e:e + 1]) if nvfp4 else mx.quantize(w[e]) for e in range(E)]
    return torch.stack([c for c, _ in q]), torch.cat([s for _, s in q]), g


def moe_call(mx, x, rows, off, codes, scales, g, **kw):
    if g is None:
        return mx.moe_matvec(x, rows, off, codes, scales, **kw)
    return mx.moe_matvec_nvfp4(x, rows, off, codes, scales, g, **kw)


def check_moe(mx, x, rows, off, codes, scales, g, total, dtype=F32):
    E, N = codes.shape[:2]
    buf = torch.full((total, N + 5), 77.0, dtype=dtype, device="cuda")
    y, st = moe_call(mx, x, rows, off, codes, scales, g, out=buf[:, :N])
    assert int(st.item()) == 0
    o = off.tolist()
    per = scales.numel() // E
    for e in range(E):
        if o[e] == o[e + 1]:
            continue
        xs = x[o[e]:o[e + 1]] if rows is None else x[rows[o[e]:o[e + 1]].long()]
        w = R.weights(codes[e], scales[e * per:(e + 1) * per], g is not None,
                      1.0 if g is None else g[e])
        want, bound = R.product(xs, w, dtype)
        R.close(y[o[e]:o[e + 1]], want, bound)
    assert (buf[o[E]:] == 77.0).all(), "wrote rows that no route fills"
    assert (buf[:, N:] == 77.0).all(), "wrote past a row of y"


MOE = [(1, 2, 8, 128, 256), (1, 1, 1, 48, 32), (5, 3, 7, 200, 96), (16, 4, 16, 130, 160),
       (40, 2, 3, 33, 288), (64, 8, 40, 256, 512), (100, 1, 2, 65, 64), (3, 3, 300, 16, 64)]


@pytest.mark.parametrize("T,k,E,N,K", MOE)
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_moe_matvec(mx, T, k, E, N, K, nvfp4, dtype):
    codes, scales, g = make_experts(mx, E, N, K, nvfp4, E + N)
    off, rows = route(mx, T, k, E, T + k + E, drop=0.2 if T > 4 else 0.0)
    check_moe(mx, rand((T, K), 3, dtype), rows, off, codes, scales, g, T * k)
    check_moe(mx, rand((T * k, K), 4, dtype), None, off, codes, scales, g, T * k, dtype)


def test_moe_matvec_uneven_segments(mx):
    E, N, K = 6, 96, 128
    codes, scales, _ = make_experts(mx, E, N, K, False, 1)
    for o in ([0, 0, 0, 0, 0, 0, 0], [0, 0, 70, 70, 71, 71, 71], [0, 100, 100, 100, 100, 100, 100],
              [0, 1, 2, 3, 36, 69, 90]):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        check_moe(mx, rand((100, K), 2), None, off, codes, scales, None, 100)


def test_moe_matvec_status(mx):
    E, N, K = 3, 40, 64
    codes, scales, _ = make_experts(mx, E, N, K, False, 1)
    x = rand((4, K), 2)
    rows = torch.tensor([0, 3, 9, 1, -1, 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 5, 6], dtype=torch.int32, device="cuda")
    y, st = mx.moe_matvec(x, rows, off, codes, scales, out_dtype=F32)
    assert int(st.item()) == mx.MXFP4_EINDEX
    assert (y[2] == 0).all() and (y[4] == 0).all()
    w = R.weights(codes[2], scales[2 * scales.numel() // 3:], False)
    want, bound = R.product(x[2:3], w, F32)
    R.close(y[5:], want, bound)
    # an index past the last row that is used does not matter
    y, st = mx.moe_matvec(x, rows, torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda"),
                          codes, scales)
    assert int(st.item()) == mx.MXFP4_OK
    for bad in ([0, 4, 2, 6], [1, 2, 5, 6], [0, 2, 5, 7], [0, -1, 5, 6]):
        y = torch.full((6, N), 3.0, dtype=BF16, device="cuda")
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        _, st = mx.moe_matvec(x, rows.abs() % 4, off, codes, scales, out=y)
        assert int(st.item()) == mx.MXFP4_EOFFSETS and (y == 3.0).all(), bad


def test_moe_matvec_offsets_past_32_bits(mx):
    """Weights of more than 2^32 bytes: the last expert's are past it."""
    E, N, K = 17, 8192, 65536
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    assert codes[E - 1].data_ptr() - codes.data_ptr() >= 2 ** 32
    per = mx.mxfp4_scale_bytes(N, K)
    scales = torch.full((E * per,), 120, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes[E - 1] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    x = rand((2, K), 3)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 2
    y, st = mx.moe_matvec(x, None, off, codes, scales, out_dtype=F32)
    assert int(st.item()) == 0
    for r in (0, 4000, 8100):
        w = R.elements(codes[E - 1, r:r + 64]) * 2.0 ** -7
        want, bound = R.product(x, w, F32)
        R.close(y[:, r:r + 64], want, bound)


def test_refusals(mx):
    codes, scales, _ = make_weights(mx, 64, 64, False, 1)
    x = rand((2, 64), 1)
    y = torch.full((2, 64), 7.0, dtype=BF16, device="cuda")
    for fn in (lambda: mx.matvec(x.float(), codes, scales, out=y),
               lambda: mx.matvec(x, codes[:, :16], scales, out=y),
               lambda: mx.matvec(x, codes, scales[:-1], out=y),
               lambda: mx.matvec(x, codes, scales, out=y[:, :63]),
               lambda: mx.matvec(x, codes, scales, out=y.to(F16)),
               lambda: mx.matvec(x.t(), codes, scales, out=y),
               lambda: mx.matvec(x.cpu(), codes, scales, out=y),
               lambda: mx.moe_matvec(x, None, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                     codes, scales, out=y),
               lambda: mx.moe_matvec(x, None, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                     codes[None], scales, out=y),
               lambda: mx.moe_matvec(x[:1], None, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                     codes[None], scales, out=y)):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(mx.MXFP4Error):                 # y over the weights
        mx.matvec(x, codes, scales, out=codes.view(-1)[:256].view(BF16).view(2, 64))
    torch.cuda.synchronize()
    assert (y == 7.0).all()

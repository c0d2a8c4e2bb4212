"""Products of 4-bit operands in the kernel's longer ways: rings of stages that go
round several times in a tile, several tiles to a CTA, experts' segments whose K is
shared by a cluster, rows wider apart than they are long; and the weighted sum's
wide path between such rows."""
import pytest
import torch

import decode_reference as R
import layer_reference as L
from test_gpu_combine import inputs
from test_gpu_gemm import BF, FP, batch, dense, experts, gen, half, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


# K: 12 or 13 stages, of which the last is not whole, and scales that end inside a word
@pytest.mark.parametrize("K", [2880, 3104])
@pytest.mark.parametrize("nv", [False, True])
def test_many_stages_many_tiles(mx, K, nv):
    for T, N, gate in ((600, 4096, None), (600, 8000, "first"), (1500, 4100, None), (1500, 8192, "second")):
        kw = dict(nv=nv, dtype=FP if T == 600 else BF, bias=True, act="silu" if gate else None, gate=gate, residual=True)
        a, b = dense(mx, T, N, K, **kw), dense(mx, T, N, K, **kw)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("gate", [None, "first", "second"])
def test_experts_with_many_stages_and_tiles(mx, nv, gate):
    g = torch.Generator().manual_seed(5)
    sizes = (torch.rand(40, generator=g) ** 3 * 700).int().tolist()
    sizes[3], sizes[11], sizes[39] = 0, 1, 0
    experts(mx, sizes, 2000, 1312, nv=nv, dtype=FP if gate else BF, bias=True, act="gelu" if gate else None, gate=gate, extra=30)
    experts(mx, [n // 20 for n in sizes], 2000, 1312, nv=nv, gate=gate, extra=3)


# fewer tiles than half the SMs and four stages or more: clusters, some without a tile
@pytest.mark.parametrize("sizes", [[3, 0, 1, 4], [0, 0, 0, 8], [1] * 8 + [0] * 20, [0, 140, 0, 5], [0, 0]])
@pytest.mark.parametrize("K", [1024, 2048, 2336])
@pytest.mark.parametrize("nv", [False, True])
def test_experts_in_clusters(mx, sizes, K, nv):
    experts(mx, sizes, 192, K, nv=nv, bias=True, act="silu", gate="second", extra=2)
    experts(mx, sizes, 330, K, nv=nv, dtype=FP)


@pytest.mark.parametrize("bad", [[1, 5, 9, 12], [0, 6, 5, 12], [0, 5, 9, 13], [0, -1, 9, 12]])
@pytest.mark.parametrize("N,gate", [(200, None), (320, "first")])
def test_bad_offsets_in_clusters(mx, bad, N, gate):
    g = gen(13)
    xc, xs, _, _, _ = batch([5, 4, 3], 2048, False, g)
    w = [operand(N, 2048, False, g) for _ in range(3)]
    y = torch.full((12, N // 2 if gate else N), 7.0, dtype=BF, device="cuda")
    _, status = mx.moe_gemm(xc, xs, torch.tensor(bad, dtype=torch.int32, device="cuda"), torch.stack([c for c, _ in w]),
                            torch.cat([s for _, s in w]), gate=gate, out=y)
    assert int(status) == mx.MXFP4_EOFFSETS and (y == 7).all()


@pytest.mark.parametrize("T,N,K,gate", [(37, 256, 64, None), (300, 640, 96, None), (130, 512, 192, "first"), (3, 256, 2048, None),
                                        (40, 512, 1024, "second")])
@pytest.mark.parametrize("pad", [64, 2, 3])
def test_rows_wider_apart_than_long(mx, T, N, K, gate, pad):
    """y, the residual, and both in one place, in rows of whole words (pad 64 and 2) and not."""
    g = gen(17)
    (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
    x, w = R.weights(xc, xs, False), R.weights(wc, ws, False)
    cols = N // 2 if gate else N
    residual = half(g, BF, T, cols + 2 * pad)[:, pad:pad + cols]
    whole = torch.full((T + 1, cols + pad), 7.0, dtype=BF, device="cuda")
    y = whole[:T, :cols]
    mx.mxfp4_gemm(xc, xs, wc, ws, y, residual=residual, gate=gate)
    want, bound = L.gemm(x, w, BF, gate=gate, residual=residual)
    L.close(y, want, bound)
    assert (whole[:, cols:] == 7).all() and (whole[T] == 7).all()
    y.copy_(residual)
    mx.mxfp4_gemm(xc, xs, wc, ws, y, residual=y, gate=gate)
    L.close(y, want, bound)
    assert (whole[:, cols:] == 7).all() and (whole[T] == 7).all()


@pytest.mark.parametrize("N,pad", [(64, 8), (2048, 64), (40, 24), (7168, 8)])
@pytest.mark.parametrize("f32", [False, True])
def test_combine_in_rows_wider_apart_than_long(mx, N, pad, f32):
    g = gen(18)
    T, k = 23, 5
    rows, dest, w = inputs(T, k, N + pad, BF, f32, g)
    rows = rows[:, 8:8 + N] if pad > 8 else rows[:, :N]
    residual = half(g, BF, T, N + 2 * pad)[:, pad:pad + N]
    whole = torch.full((T + 1, N + pad), 7.0, dtype=BF, device="cuda")
    y = whole[:T, :N]
    want, bound = L.combine(rows, dest, w, BF, residual)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    mx.mxfp4_moe_combine(rows, dest, w, y, residual=residual, status=status)
    R.close(y, want, bound)
    y.copy_(residual)
    mx.mxfp4_moe_combine(rows, dest, w, y, residual=y)
    R.close(y, want, bound)
    assert int(status) == 0 and (whole[:, N:] == 7).all() and (whole[T] == 7).all()


def test_outputs_past_32_bit_offsets(mx):
    """More than 2^32 bytes of y (and of the residual, which is y)."""
    g = gen(19)
    T, N, K = 310_000, 7200, 64
    (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
    y = torch.ones(T, N, dtype=BF, device="cuda")
    mx.mxfp4_gemm(xc, xs, wc, ws, y, residual=y)
    w = R.weights(wc, ws, False)
    for lo, hi in ((0, 40), (149_100, 149_160), (298_200, 298_300), (T - 150, T)):
        flat = R.untile(xs[lo // 128 * 512:], hi - lo // 128 * 128, 2)[lo % 128:]
        x = R.rows_of(xc[lo:hi], flat, False)
        L.close(y[lo:hi], *L.gemm(x, w, BF, residual=torch.ones(hi - lo, N, device="cuda")))
    del y


def test_weights_past_32_bit_offsets(mx):
    """More than 2^32 bytes of the experts' codes: rows of the first and the last ones."""
    g = gen(20)
    E, N, K = 130, 8192, 8192
    sizes = [0] * E
    sizes[0], sizes[127], sizes[128], sizes[129] = 3, 2, 1, 140
    xc, xs, off, values, _ = batch(sizes, K, False, g)
    codes = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((E * N * K // 32,), 127, dtype=torch.uint8, device="cuda")
    per, used = N * K // 32, [e for e, n in enumerate(sizes) if n]
    for e in used:
        codes[e], scales[e * per:(e + 1) * per] = operand(N, K, False, g)
    y, status = mx.moe_gemm(xc, xs, off, codes, scales)
    assert int(status) == 0
    at = 0
    for e, x in zip(used, values):
        part = slice(0, 200) if e == 129 else slice(0, N)
        w = R.weights(codes[e], scales[e * per:(e + 1) * per], False)
        want, bound = L.gemm(x, w[part], BF)
        L.close(y[at:at + sizes[e], part], want, bound)
        at += sizes[e]

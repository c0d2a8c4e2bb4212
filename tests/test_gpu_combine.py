"""The experts' rows back to their tokens against the 64-bit form."""
import pytest
import torch

import decode_reference as R
import layer_reference as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def inputs(T, k, N, dtype, f32, g, rows=None, drop=0.2):
    rows = T * k if rows is None else rows
    data = torch.randn(rows, N, device="cuda", generator=g).to(torch.float32 if f32 else dtype)
    dest = torch.randint(0, max(rows, 1), (T, k), device="cuda", generator=g)
    dest[torch.rand(T, k, device="cuda", generator=g) < drop] = -1
    if rows == 0:
        dest[:] = -1
    return data, dest.to(torch.int32), torch.randn(T, k, device="cuda", generator=g)


@pytest.mark.parametrize("T,k,N", [(1, 8, 7168), (1, 1, 1), (3, 2, 7), (5, 4, 8), (33, 3, 64), (7, 5, 1000), (40, 9, 2048),
                                   (300, 8, 40), (2, 32, 2056), (1000, 1, 8), (4, 6, 2047), (3, 7, 20000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("f32", [False, True])
def test_sizes(mx, T, k, N, dtype, f32):
    g = gen(T + k + N)
    rows, dest, w = inputs(T, k, N, dtype, f32, g)
    r = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    for residual in (None, r):
        y, status = mx.moe_combine(rows, dest, w, residual=residual, out_dtype=dtype)
        assert int(status) == 0
        R.close(y, *L.combine(rows, dest, w, dtype, residual))
    mx.mxfp4_moe_combine(rows, dest, w, y, residual=y)        # added to what is there
    R.close(y, *L.combine(rows, dest, w, dtype, L_rounded(rows, dest, w, r)))


def L_rounded(rows, dest, w, r):
    import mxfp4_block_quantization_gb300 as m
    return m.moe_combine(rows, dest, w, residual=r)[0]


def test_routes_that_add_nothing(mx):
    """-1 everywhere, weights of NaN there, rows of infinities that no route takes."""
    g = gen(1)
    rows, dest, w = inputs(9, 3, 40, torch.bfloat16, False, g, drop=0.0)
    dest[4] = -1
    dest[5, 1:] = -1
    w[4], w[5, 1:] = float("nan"), float("inf")
    taken = torch.zeros(27, dtype=torch.bool, device="cuda")
    taken[dest[dest >= 0].long()] = True
    rows[~taken] = float("inf")
    y, status = mx.moe_combine(rows, dest, w)
    assert int(status) == 0 and (y[4] == 0).all() and torch.isfinite(y).all()
    want, bound = L.combine(rows.nan_to_num(posinf=0.0), dest, w.nan_to_num(0.0, 0.0), torch.bfloat16)
    R.close(y, want, bound)
    none = torch.zeros(0, 40, dtype=torch.bfloat16, device="cuda")
    y, status = mx.moe_combine(none, torch.full((9, 3), -1, dtype=torch.int32, device="cuda"), w)
    assert int(status) == 0 and (y == 0).all()


@pytest.mark.parametrize("bad", [-2, 27, 2 ** 31 - 1, -2 ** 31])
def test_bad_entries(mx, bad):
    g = gen(2)
    rows, dest, w = inputs(9, 3, 48, torch.float16, False, g)
    dest[7, 2] = bad
    y, status = mx.moe_combine(rows, dest, w)
    assert int(status) == mx.MXFP4_EINDEX
    R.close(y, *L.combine(rows, dest, w, torch.float16))


def test_strides_and_places(mx):
    g = gen(3)
    T, k = 13, 4
    for N, ld, first in ((40, 48, 8), (40, 41, 1), (33, 64, 0), (64, 72, 4)):
        rows = torch.randn(52, ld, device="cuda", generator=g).to(torch.bfloat16)[:, first:first + N] if first + N <= ld else \
            torch.randn(52, ld, device="cuda", generator=g).to(torch.bfloat16)[:, :N]
        _, dest, w = inputs(T, k, N, torch.bfloat16, False, g)
        whole = torch.full((T, ld + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        residual = torch.randn(T, ld, device="cuda", generator=g).to(torch.bfloat16)[:, :N]
        mx.mxfp4_moe_combine(rows, dest, w, whole[:, 1:1 + N], residual=residual)
        R.close(whole[:, 1:1 + N], *L.combine(rows, dest, w, torch.bfloat16, residual))
        assert (whole[:, 0] == 7).all() and (whole[:, 1 + N:] == 7).all()


def test_rows_past_32_bit_offsets(mx):
    """More than 2^32 bytes of rows."""
    rows = torch.zeros(300_000, 7200, dtype=torch.bfloat16, device="cuda")
    rows[299_999], rows[149_131], rows[1] = 1.0, 2.0, 4.0
    dest = torch.tensor([[299_999, 149_131], [1, 2]], dtype=torch.int32, device="cuda")
    y, status = mx.moe_combine(rows, dest, torch.tensor([[1.0, 0.5], [0.25, 9.0]], device="cuda"))
    assert int(status) == 0 and (y[0] == 2).all() and (y[1] == 1).all()


def test_empty(mx):
    rows = torch.zeros(4, 0, dtype=torch.bfloat16, device="cuda")
    dest = torch.tensor([[0, 1], [3, 9]], dtype=torch.int32, device="cuda")
    y, status = mx.moe_combine(rows, dest, torch.ones(2, 2, device="cuda"))
    assert y.shape == (2, 0) and int(status) == mx.MXFP4_EINDEX
    y, status = mx.moe_combine(torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"), dest[:0], torch.ones(0, 2, device="cuda"))
    assert y.shape == (0, 8) and int(status) == 0


def test_refusals(mx):
    g = gen(4)
    rows, dest, w = inputs(6, 2, 16, torch.bfloat16, False, g)
    with pytest.raises(ValueError, match="y must"):
        mx.mxfp4_moe_combine(rows, dest, w, torch.empty(5, 16, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="rows"):
        mx.moe_combine(rows, dest, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="weights"):
        mx.moe_combine(rows, dest, w.double())
    with pytest.raises(ValueError, match="dest_rows"):
        mx.moe_combine(rows, dest.flatten(), w)
    with pytest.raises(ValueError, match="residual"):
        mx.moe_combine(rows, dest, w, residual=rows)
    with pytest.raises(mx.MXFP4Error):
        mx.mxfp4_moe_combine(rows, dest, w, rows[:6])

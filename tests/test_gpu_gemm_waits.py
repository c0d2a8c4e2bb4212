"""Products one of whose CTAs never gets what it waits for: the waits run out after
about two seconds, that CTA's tiles are NaN and nothing else is touched, the experts'
calls say so in their status word, and the next call is right again.  In the
bounds-checking build, which can hold one role of the last CTA back."""
import pytest
import torch

import decode_reference as R
import layer_reference as L
from test_gpu_decode_bounds import libs, using  # noqa: F401
from test_gpu_gemm import BF, FP, batch, gen, half, operand

pytestmark = pytest.mark.gpu

TILES, COPIES, PRODUCTS = 1, 2, 3


class Held:
    """The debug library in place of the normal one, `role` held back."""

    def __init__(self, libs, role):
        self.mx, _, self.dbg = libs
        self.role, self.using = role, using(self.mx, self.dbg)

    def __enter__(self):
        self.using.__enter__()
        assert self.dbg.mxfp4_debug_stall_products(self.role) == 0

    def __exit__(self, *e):
        assert self.dbg.mxfp4_debug_stall_products(0) == 0
        self.using.__exit__(*e)
        assert self.dbg.mxfp4_debug_bounds_violations() == 0


@pytest.mark.parametrize("role", [TILES, COPIES, PRODUCTS])
# the last tile's weights and tokens: alone (96 tiles of 256 tokens), one of many (its
# CTA has the tiles 151 and 303 of 320), and shared by a cluster
@pytest.mark.parametrize("T,N,K,gate,lost", [(600, 4096, 288, None, [(512, 3968)]), (1024, 10240, 64, "first", [(896, 2304), (896, 4736)]),
                                             (5, 130, 7168, None, [(0, 128)])])
def test_dense(libs, role, T, N, K, gate, lost):  # noqa: F811
    g = gen(31)
    (xc, xs), (wc, ws) = operand(T, K, False, g), operand(N, K, False, g)
    cols = N // 2 if gate else N
    old = half(g, BF, T, cols)
    want, bound = L.gemm(R.weights(xc, xs, False), R.weights(wc, ws, False), BF, gate=gate, residual=old)
    whole = torch.full((T + 1, cols + 4), 7.0, dtype=BF, device="cuda")
    y = whole[:T, :cols]
    tokens = 128 if gate else 256
    there = torch.ones(T, cols, dtype=torch.bool, device="cuda")
    for t, n in lost:
        there[t:t + tokens, n:n + 128] = False
    y.copy_(old)
    with Held(libs, role):
        libs[0].mxfp4_gemm(xc, xs, wc, ws, y, residual=y, gate=gate)
    assert torch.isnan(y[~there]).all()
    L.close(y[there], want[there], bound[there])
    assert (whole[:, cols:] == 7).all() and (whole[T] == 7).all()
    y.copy_(old)
    libs[0].mxfp4_gemm(xc, xs, wc, ws, y, residual=y, gate=gate)
    L.close(y, want, bound)


@pytest.mark.parametrize("role", [TILES, COPIES, PRODUCTS])
# 192 tiles (K's scales to be mended), of which the last CTA has one; and clusters, the last of which has none
@pytest.mark.parametrize("sizes,N,K,all_there", [([100, 0, 300], 8192, 96, False), ([3, 0, 1, 4], 192, 2048, True)])
def test_experts(libs, role, sizes, N, K, all_there):  # noqa: F811
    mx, g, E = libs[0], gen(32), len(sizes)
    xc, xs, off, values, xg = batch(sizes, K, True, g, extra=2)
    w = [operand(N, K, True, g) for _ in range(E)]
    wc, ws, wg = torch.stack([c for c, _ in w]), torch.cat([s for _, s in w]), torch.full((E,), 2.0, device="cuda")
    y = torch.full((sum(sizes) + 2, N), 7.0, dtype=FP, device="cuda")

    def call():
        return mx.moe_gemm_nvfp4(xc, xs, xg, off, wc, ws, wg, out=y)[1]

    def check(nan):
        at, live, seen = 0, iter(values), 0
        for e, n in enumerate(sizes):
            if n:
                want, bound = L.gemm(next(live), R.weights(wc[e], w[e][1], True, wg[e]), FP)
                lost = torch.isnan(y[at:at + n])
                L.close(y[at:at + n][~lost], want[~lost], bound[~lost])
                seen += int(lost.sum())
                at += n
        assert (y[at:] == 7).all()
        assert seen == 0 if not nan else 0 < seen <= 256 * 128

    with Held(libs, role):
        status = call()
    # with no tile to find, the last cluster misses the word that there is none
    assert int(status) == (mx.MXFP4_OK if all_there and role != TILES else mx.MXFP4_ECUDA)
    check(not all_there)
    assert int(call()) == 0
    check(False)

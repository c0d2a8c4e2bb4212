"""Products and attention within bounds that a lost block is outside of (see
decode_sums), up to contexts of 131072 positions."""
import pytest
import torch

import decode_reference as R
import decode_sums as S
from test_gpu_attention_edges import contents
from test_gpu_attention_split import with_room
from test_gpu_cache import BF16, F16, filled, mx, rand, tables  # noqa: F401
from test_gpu_matvec import F32, call, make_experts, make_weights, moe_call, route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(1, 640, 16384), (4, 300, 7168), (16, 1000, 7168), (9, 200, 2880), (1, 129, 768),
                                   (33, 256, 2048)])
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_products(mx, T, N, K, nvfp4, dtype):  # noqa: F811
    codes, scales, g = make_weights(mx, N, K, nvfp4, N + K)
    x = rand((T, K), T + K, dtype)
    w = R.weights(codes, scales, g is not None, 1.0 if g is None else g)
    R.close(call(mx, x, codes, scales, g, out_dtype=F32), *S.product(x, w, F32))


@pytest.mark.parametrize("nvfp4", [False, True])
def test_experts(mx, nvfp4):  # noqa: F811
    E, N, K = 12, 200, 4096
    codes, scales, g = make_experts(mx, E, N, K, nvfp4, 1)
    off, rows = route(mx, 50, 3, E, 4)
    x = rand((50, K), 3)
    y, _ = moe_call(mx, x, rows, off, codes, scales, g, out_dtype=F32)
    o, per = off.tolist(), scales.numel() // E
    for e in range(E):
        w = R.weights(codes[e], scales[e * per:(e + 1) * per], nvfp4, 1.0 if g is None else g[e])
        R.close(y[o[e]:o[e + 1]], *S.product(x[rows[o[e]:o[e + 1]].long()], w, F32))


@pytest.mark.parametrize("n,Hq,H,D,S_", [(300, 8, 2, 64, 16), (700, 64, 8, 128, 16), (12000, 8, 1, 64, 128),
                                         (12000, 16, 1, 128, 24), (131072, 8, 1, 64, 32), (131071, 4, 2, 128, 64),
                                         (65537, 3, 1, 256, 48)])
@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("room", [False, True])
def test_attention(mx, n, Hq, H, D, S_, nvfp4, room):  # noqa: F811
    pages = -(-n // S_)
    c = filled(mx, pages, S_, H, D, nvfp4, 7, F16)
    table = tables(1, pages, pages, 2)
    q = rand((1, Hq, D), 5, F16)
    o, _, st = mx.cache_attention(q, c, with_room(table, S_, 140000) if room else table,
                                  torch.tensor([n], dtype=torch.int32, device="cuda"), D ** -0.5)
    assert int(st.item()) == 0
    k, v = contents(c, table[0].long(), n)
    G = Hq // H
    for h in range(H):
        R.close(o[0, h * G:(h + 1) * G], *S.attention(q[0, h * G:(h + 1) * G], k[h], v[h], D ** -0.5, F16))

"""Attention over the paged 4-bit cache where the same contexts are split
differently: a table with room for far more positions than there are makes the
call share all steps among the GPU's warps and join the parts in a second
kernel; a table of just the pages leaves each context to a cluster."""
import pytest
import torch

from test_gpu_cache import BF16, F16, SHAPES, check_attention, filled, mx, rand, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def with_room(table, S, positions=40000):
    wide = torch.full((table.shape[0], positions // S), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("lens,Hq,H,D,S", SHAPES)
@pytest.mark.parametrize("nvfp4", [False, True])
def test_room_for_more(mx, lens, Hq, H, D, S, nvfp4):  # noqa: F811
    dtype = F16 if nvfp4 else BF16
    B, per = len(lens), -(-max(lens) // S)
    c = filled(mx, per * 2 + 1, S, H, D, nvfp4, D + S, dtype)
    table = with_room(tables(B, per, per * 2 + 1, 3), S)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = rand((B, Hq, D), 5, dtype)
    check_attention(mx, q, c, table, n, D ** -0.5)
    check_attention(mx, q, c, table, n, 1.1, window=40)
    check_attention(mx, q, c, table, torch.zeros_like(n), 1.0)


@pytest.mark.parametrize("positions", [33, 128, 129, 257, 1024, 1025, 4096, 8192, 8193])
@pytest.mark.parametrize("B,H,D", [(1, 1, 64), (3, 2, 128), (40, 8, 32), (2, 1, 256)])
def test_room_by_room(mx, positions, B, H, D):  # noqa: F811
    S = 16
    c = filled(mx, 600, S, H, D, False, 3)
    per = -(-positions // S)
    lens = torch.randint(0, positions + 1, (B,), generator=torch.Generator().manual_seed(positions))
    lens[0] = positions
    check_attention(mx, rand((B, 3 * H, D), 7), c, tables(B, per, 600, 2), lens.int().cuda(), 0.1)


@pytest.mark.parametrize("window", [1, 17, 64, 1000, 5000])
def test_windows_with_room(mx, window):  # noqa: F811
    c = filled(mx, 70, 16, 2, 64, False, 9)
    n = torch.tensor([1000, 16, 65, 0, 1], dtype=torch.int32, device="cuda")
    check_attention(mx, rand((5, 8, 64), 4), c, with_room(tables(5, 64, 70, 1), 16), n, 0.3, window=window)


@pytest.mark.parametrize("S,room", [(16, None), (16, 40000), (1, None), (100, 40000)])
def test_status_of_many(mx, S, room):  # noqa: F811
    """One page out of range anywhere, inside a length or past it; and one length."""
    B, per = 150, 3
    c = filled(mx, 6, S, 1, 64, False, 4)
    table = tables(B, per, 6, 1)
    if room:
        table = with_room(table, S, room)
    n = torch.randint(0, per * S + 1, (B,), device="cuda", dtype=torch.int32)
    n[7], n[149] = 2 * S, 2 * S + 1
    q = rand((B, 2, 64), 5)

    def status():
        return int(mx.cache_attention(q, c, table, n, 0.2)[2].item())

    assert status() == mx.MXFP4_OK
    for b, i, page, want in ((7, 2, 6, mx.MXFP4_OK), (7, 1, 6, mx.MXFP4_EINDEX), (149, 2, -1, mx.MXFP4_EINDEX)):
        keep = int(table[b, i])
        table[b, i] = page
        assert status() == want
        table[b, i] = keep
    for b, length in ((0, -1), (149, table.shape[1] * S + 1)):
        keep = int(n[b])
        n[b] = length
        assert status() == mx.MXFP4_EINDEX
        n[b] = keep


def test_same_bits_with_room(mx):  # noqa: F811
    c = filled(mx, 300, 16, 2, 128, False, 4)
    q, table = rand((2, 16, 128), 5), with_room(tables(2, 256, 300, 1), 16)
    n = torch.tensor([4096, 3001], dtype=torch.int32, device="cuda")
    o, lse, _ = mx.cache_attention(q, c, table, n, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [mx.cache_attention(q, c, table, n, 0.1, stream=s) for _ in range(4)]
    s.synchronize()
    for a, b, _ in got:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_masked_bytes_with_room(mx):  # noqa: F811
    S, H, D = 16, 2, 128
    for nvfp4, nan in ((False, 255), (True, 0x7F)):
        c = filled(mx, 12, S, H, D, nvfp4, 1)
        n = torch.tensor([37, 5, 0], dtype=torch.int32, device="cuda")
        table = torch.tensor([[3, 7, 1, -5], [9, 10 ** 9, -1, 4], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda")
        live = torch.zeros(12, S, dtype=torch.bool, device="cuda")
        live[3], live[7], live[1, :5], live[9, :5] = True, True, True, True
        for t in (c.k_scales, c.v_scales):
            t.transpose(1, 2)[~live] = nan
        check_attention(mx, rand((3, 16, D), 2), c, with_room(table, S), n, 0.1)


@pytest.mark.parametrize("group", [9, 16, 17, 31, 64])
@pytest.mark.parametrize("H,D,S", [(1, 128, 16), (2, 64, 7), (1, 32, 64), (3, 96, 16), (1, 256, 32)])
@pytest.mark.parametrize("nvfp4,dtype", [(False, BF16), (True, F16)])
def test_more_heads_than_a_block(mx, group, H, D, S, nvfp4, dtype):  # noqa: F811
    lens = [700, 0, 33, 1]
    per = -(-max(lens) // S)
    c = filled(mx, 2 * per, S, H, D, nvfp4, group, dtype)
    table = tables(len(lens), per, 2 * per, 3)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = rand((len(lens), group * H, D), 5, dtype)
    check_attention(mx, q, c, table, n, D ** -0.5)
    check_attention(mx, q, c, with_room(table, S, 70000), n, -0.7, window=300)


@pytest.mark.parametrize("B,group,D,L,nvfp4", [(400, 16, 32, 320, False), (300, 13, 128, 352, True),
                                               (290, 16, 128, 352, False), (150, 24, 64, 1700, False)])
def test_more_heads_in_clusters(mx, B, group, D, L, nvfp4):  # noqa: F811
    """Many sequences of few steps, more than 8 heads to a kv head."""
    S, pages = 16, 400
    c = filled(mx, pages, S, 1, D, nvfp4, 6)
    lens = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(L)).int().cuda()
    lens[0] = L
    check_attention(mx, rand((B, group, D), 7), c, tables(B, -(-L // S), pages, 2), lens, 0.1)


@pytest.mark.parametrize("power", [-100, -60, -20, 0])
@pytest.mark.parametrize("scale", [0.0, 1e-25, -1e-3])
@pytest.mark.parametrize("room", [False, True])
def test_small_queries_and_scales(mx, power, scale, room):  # noqa: F811
    """Scores that all but vanish, beside masked positions."""
    c = filled(mx, 8, 16, 1, 64, False, 6)
    n = torch.tensor([100, 33, 1], dtype=torch.int32, device="cuda")
    q = (rand((3, 4, 64), 5).float() * 2.0 ** power).to(BF16)
    table = tables(3, 7, 8, 1)
    check_attention(mx, q, c, with_room(table, 16) if room else table, n, scale)


@pytest.mark.parametrize("scale", [0.2, -0.2])
def test_negative_global_scale(mx, scale):  # noqa: F811
    c = filled(mx, 8, 16, 2, 64, True, 6)
    c = c._replace(k_global=-c.k_global)
    n = torch.tensor([100, 33, 0], dtype=torch.int32, device="cuda")
    check_attention(mx, rand((3, 8, 64), 5), c, tables(3, 7, 8, 1), n, scale)

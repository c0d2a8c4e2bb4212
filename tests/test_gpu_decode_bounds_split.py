"""The bounds-checking build where the attention's contexts are shared by all warps:
parts in the workspace and in the CTAs' rings, each form of the joining kernel,
units of 16 heads, and the status word alone; and the products' and the cache's
calls with their index tensors at the ends of a buffer."""
import pytest
import torch

from test_gpu_attention_split import with_room
from test_gpu_decode_bounds import check, libs, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def cache_of(mx, pages, S, H, D, nvfp4):
    g = (torch.tensor([300.0], device="cuda"),) * 2 if nvfp4 else ()
    c = mx.cache_alloc(pages, S, H, D, *g)
    n = pages * S
    mx.cache_write(rand((n, H, D), 1), rand((n, H, D), 2), torch.arange(n, dtype=torch.int32, device="cuda"), c)
    return c


# sequences, query heads to a kv head, kv heads, head_dim, page size, longest length,
# positions that the table has room for
SHARED = [(1, 1, 1, 64, 16, 9000, 40000), (1, 8, 1, 128, 7, 30000, 30100), (4, 3, 2, 96, 24, 2500, 40000),
          (110, 8, 4, 64, 16, 700, 4000), (300, 1, 2, 32, 5, 100, 40000), (40, 16, 4, 128, 16, 900, 4000),
          (2, 20, 1, 64, 32, 3000, 70000), (3, 4, 1, 256, 16, 5000, 40000), (9, 2, 1, 224, 11, 2000, 9000)]


@pytest.mark.parametrize("B,group,H,D,S,L,room", SHARED)
@pytest.mark.parametrize("nvfp4", [False, True])
def test_shared_steps_in_bounds(libs, B, group, H, D, S, L, room, nvfp4):  # noqa: F811
    mx = libs[0]
    pages = max(64, L // S + 1)
    c = cache_of(mx, pages, S, H, D, nvfp4)
    gen = torch.Generator(device="cuda").manual_seed(B + L)
    per = -(-L // S)
    table = torch.randint(0, pages, (B, per), generator=gen, device="cuda").to(torch.int32)
    lens = torch.randint(0, L + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    lens[0] = L
    if B > 2:
        lens[1], lens[2] = 0, -3                       # empty; out of range
        table[B - 1, 0] = pages
    wide = with_room(table, S, room)
    q = rand((B, group * H, D), 3)
    assert mx.mxfp4_cache_attention_workspace_bytes(B, group * H, H, D, S, wide.shape[1]) > 0

    def call(window, status=True):
        out = torch.zeros((B, group * H, D), dtype=q.dtype, device="cuda")
        need = mx.mxfp4_cache_attention_workspace_bytes(B, group * H, H, D, S, wide.shape[1])
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")       # just what the call asks for
        lse = torch.zeros((B, group * H), dtype=torch.float32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
        mx.mxfp4_cache_attention(q, c, wide, lens, 0.1, out, window, ws, lse if status else None, st)
        return (out, lse, st) if status else (out,)

    check(libs, lambda: call(0))
    check(libs, lambda: call(50))
    check(libs, lambda: call(0, status=False))


def test_status_alone_in_bounds(libs):  # noqa: F811
    mx = libs[0]
    c = cache_of(mx, 6, 16, 1, 64, False)
    table = torch.tensor([[0, 1, 5], [2, 6, 0]], dtype=torch.int32, device="cuda")
    q = torch.empty((2, 0, 64), dtype=torch.bfloat16, device="cuda")
    for lens, want in (([48, 16], mx.MXFP4_OK), ([48, 17], mx.MXFP4_EINDEX), ([49, 0], mx.MXFP4_EINDEX)):
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        check(libs, lambda: (mx.cache_attention(q, c, table, n, 0.1)[2],))
        assert int(mx.cache_attention(q, c, table, n, 0.1)[2].item()) == want


def test_indexes_in_bounds(libs):  # noqa: F811
    """Offsets, row indexes and slots that fill their tensors exactly, many experts."""
    mx = libs[0]
    E, N, K, rows = 600, 16, 64, 700
    w = mx.quantize(rand((N, K), 1))
    codes, scales = w[0].repeat(E, 1, 1), w[1].repeat(E)
    cuts = torch.sort(torch.randint(0, rows + 1, (E - 1,), device="cuda")).values.to(torch.int32)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.cat((zero, cuts, zero + rows))
    index = torch.randint(0, 50, (rows,), device="cuda").to(torch.int32)
    x = rand((50, K), 2)
    check(libs, lambda: mx.moe_matvec(x, index, off, codes, scales))
    c = mx.cache_alloc(3, 7, 2, 32)
    slots = torch.randperm(21, device="cuda").to(torch.int32)
    kv = rand((21, 2, 2, 32), 4)

    def write():
        st = mx.cache_write(kv[:, 0], kv[:, 1], slots, c)
        return (*c[:4], st, *mx.cache_read(c, slots))

    check(libs, write)

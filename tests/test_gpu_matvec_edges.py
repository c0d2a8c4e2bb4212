"""Products with 4-bit weights where bytes that are no weight's lie beside the weights',
and empty sums."""
import pytest
import torch

from test_gpu_matvec import BF16, F16, F32, make_experts, make_weights, moe_call, call, mx, rand, route  # noqa: F401

pytestmark = pytest.mark.gpu


def pad_bytes(rows, cols, device="cuda"):
    """Mask of a tiled scale buffer: the bytes that are no (row, column)'s."""
    mt, kt = -(-rows // 128), -(-cols // 4)
    used = torch.zeros(mt * kt * 512, dtype=torch.bool, device=device)
    r = torch.arange(rows, device=device).view(-1, 1)
    c = torch.arange(cols, device=device)
    used[((r // 128) * kt + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = True
    return ~used


SIZES = [(1, 130, 96), (3, 200, 160), (9, 40, 288), (1, 300, 2880), (16, 129, 2880), (5, 64, 736), (17, 33, 1056)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("nvfp4,byte", [(False, 255), (True, 0x7F), (True, 0xFF)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_unused_scale_bytes_never_matter(mx, T, N, K, nvfp4, byte, dtype):  # noqa: F811
    codes, scales, g = make_weights(mx, N, K, nvfp4, T + N + K)
    x = rand((T, K), T + K, dtype)
    want = call(mx, x, codes, scales, g, out_dtype=F32)
    scales[pad_bytes(N, K // (16 if nvfp4 else 32))] = byte
    assert torch.equal(call(mx, x, codes, scales, g, out_dtype=F32), want)


@pytest.mark.parametrize("T,N,K", [(1, 100, 16), (4, 130, 48), (9, 31, 80), (2, 1000, 2896)])
def test_unused_scale_bytes_of_odd_blocks(mx, T, N, K):  # noqa: F811
    codes, scales, g = make_weights(mx, N, K, True, K)
    x = rand((T, K), K + 1)
    want = call(mx, x, codes, scales, g, out_dtype=F32)
    scales[pad_bytes(N, K // 16)] = 0x7F
    assert torch.equal(call(mx, x, codes, scales, g, out_dtype=F32), want)


@pytest.mark.parametrize("T,k,E,N,K", [(1, 2, 8, 130, 96), (40, 2, 3, 33, 288), (64, 4, 20, 256, 736)])
@pytest.mark.parametrize("nvfp4,byte", [(False, 255), (True, 0x7F)])
def test_unused_scale_bytes_of_experts(mx, T, k, E, N, K, nvfp4, byte):  # noqa: F811
    codes, scales, g = make_experts(mx, E, N, K, nvfp4, E + N)
    off, rows = route(mx, T, k, E, T + k + E)
    x = rand((T, K), 3)
    want, _ = moe_call(mx, x, rows, off, codes, scales, g, out_dtype=F32)
    scales[pad_bytes(N, K // (16 if nvfp4 else 32)).repeat(E)] = byte
    got, _ = moe_call(mx, x, rows, off, codes, scales, g, out_dtype=F32)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [3, 12])
def test_an_empty_sum_is_zero_nvfp4(mx, dtype, T):  # noqa: F811
    """Without elements the global scale has no say either, nor one of the call before."""
    codes, scales, _ = make_weights(mx, 5000, 64, True, 3)
    empty = torch.empty((400, 0), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for before in (float("nan"), float("inf"), -1.0):
        g = torch.tensor([before], device="cuda")
        mx.matvec_nvfp4(rand((T, 64), 1, dtype), codes, scales, g)
        x = torch.empty((T, 0), dtype=dtype, device="cuda")
        y = torch.full((T, 400), 5.0, dtype=F32, device="cuda")
        mx.matvec_nvfp4(x, empty, none, g, out=y)
        assert torch.equal(y.view(torch.int32), torch.zeros_like(y, dtype=torch.int32))
        y = torch.full((T, 400), 5.0, dtype=F32, device="cuda")
        off = torch.tensor([0, 1, T], dtype=torch.int32, device="cuda")
        mx.moe_matvec_nvfp4(x, None, off, torch.empty((2, 400, 0), dtype=torch.uint8, device="cuda"), none,
                            g.repeat(2), out=y)
        assert torch.equal(y.view(torch.int32), torch.zeros_like(y, dtype=torch.int32))

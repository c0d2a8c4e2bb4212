"""Many tokens written to and read from the paged 4-bit cache in one call: each
thread takes several, with and without a status word, bit for bit against the
dense quantizers."""
import pytest
import torch

from test_gpu_cache import BF16, F16, flat_quantized, make_cache, mx, place, rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,D,S", [(100003, 1, 32, 16), (9001, 3, 96, 7), (4099, 17, 128, 64), (20000, 2, 64, 1)])
@pytest.mark.parametrize("nvfp4,dtype", [(False, BF16), (True, F16)])
@pytest.mark.parametrize("with_status", [False, True])
def test_many_tokens(mx, T, H, D, S, nvfp4, dtype, with_status):  # noqa: F811
    pages = -(-T // S) + 1
    c = make_cache(mx, pages, S, H, D, nvfp4, fill=0xA5)
    slots = torch.randperm(pages * S, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))[:T]
    slots = slots.to(torch.int32)
    slots[::1000] = -1
    k, v = rand((T, H, D), T, dtype), rand((T, H, D), T + 1, dtype)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    mx.mxfp4_cache_write(k, v, slots, c, status if with_status else None)
    assert int(status.item()) == (0 if with_status else 9)
    live = slots >= 0
    page, at = place(slots[live], S)
    k2, v2 = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    mx.mxfp4_cache_read(c, slots, k2, v2, status if with_status else None)
    for x, got, codes, scales, g in ((k, k2, c.k_codes, c.k_scales, c.k_global),
                                     (v, v2, c.v_codes, c.v_scales, c.v_global)):
        want_c, want_s = flat_quantized(mx, x[live].reshape(-1, D), nvfp4, g)
        n = int(live.sum())
        assert torch.equal(codes[page, :, at], want_c.view(n, H, -1))
        assert torch.equal(scales[page, :, at], want_s.view(n, H, -1))
        assert (got[~live] == 0).all()
        if dtype == BF16:
            y = mx.dequantize(*mx.quantize(x[live].reshape(-1, D)), n * H, D)
            assert torch.equal(got[live].view(torch.int16), y.view(n, H, D).view(torch.int16))
    slots[T // 2] = pages * S
    mx.mxfp4_cache_write(k, v, slots, c, status)
    assert int(status.item()) == mx.MXFP4_EINDEX

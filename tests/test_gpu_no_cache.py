"""NVFP4 cache calls that touch no cache (no pages, no tokens, no room for a
position) may have no global scales, and give what empty ones give."""
import ctypes
import math

import pytest
import torch

from test_gpu_cache import BF16, F16, mx, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def at(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("tail,dtype", [("", BF16), ("_f16", F16)])
@pytest.mark.parametrize("T", [0, 5])
@pytest.mark.parametrize("with_status", [False, True])
def test_write_and_read_without_a_cache(mx, tail, dtype, T, with_status):  # noqa: F811
    H, D, S = 2, 64, 16
    k, v = rand((5, H, D), 1, dtype), rand((5, H, D), 2, dtype)
    slots = torch.tensor([-1, 0, 3, -1, 7], dtype=torch.int32, device="cuda")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    word = at(status) if with_status else None
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    L = mx._lib
    rc = getattr(L, "mxfp4_cache_write_nvfp4" + tail)(at(k), at(v), T, H, D, H * D, D, H * D, D, at(slots), 0, S, None,
                                                      None, None, None, None, None, word, stream)
    assert rc == mx.MXFP4_OK
    want = mx.MXFP4_EINDEX if T else mx.MXFP4_OK
    assert int(status.item()) == (want if with_status else 9)
    k2, v2 = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    rc = getattr(L, "mxfp4_cache_read_nvfp4" + tail)(None, None, None, None, None, None, 0, S, H, D, at(slots), T,
                                                     at(k2), at(v2), word, stream)
    assert rc == mx.MXFP4_OK
    assert (k2[:T] == 0).all() and (v2[:T] == 0).all() and (k2[T:] == 7).all()
    assert int(status.item()) == (want if with_status else 9)


@pytest.mark.parametrize("tail,dtype", [("", BF16), ("_f16", F16)])
@pytest.mark.parametrize("max_pages", [0, 2, 2000])
def test_attention_without_a_cache(mx, tail, dtype, max_pages):  # noqa: F811
    B, Hq, H, D, S = 3, 8, 2, 64, 16
    q = rand((B, Hq, D), 1, dtype)
    out = torch.full((B, Hq, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((B, Hq), 7.0, device="cuda")
    table = torch.zeros((B, max(max_pages, 1)), dtype=torch.int32, device="cuda")
    need = mx.mxfp4_cache_attention_workspace_bytes(B, Hq, H, D, S, max_pages)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for lens, want in (([0, 0, 0], mx.MXFP4_OK), ([0, 5, 0], mx.MXFP4_EINDEX)):
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        rc = getattr(mx._lib, "mxfp4_cache_attention_nvfp4" + tail)(
            at(q), B, Hq, D, Hq * D, D, None, None, None, None, None, None, 0, S, H, at(table), max(max_pages, 1),
            max_pages, at(n), 0.1, 0, at(ws), need, at(out), at(lse), at(status), stream)
        assert rc == mx.MXFP4_OK
        assert int(status.item()) == want
        assert (out == 0).all() and (lse == -math.inf).all()

"""GB300 (sm_103a) MXFP4 block quantization.

Thin Python binding of ``libmxfp4_gb300.so`` (C ABI declared in
``include/mxfp4.h``).  The functions named ``mxfp4_*`` mirror the C entry
points one to one and only marshal arguments (device pointers, sizes, the
current CUDA stream); every step of the computation runs in the library's
CUDA kernels.  ``quantize``, ``quantize_grouped``, ``dequantize`` and
``swap_w13`` are conveniences that allocate the outputs with torch and call
the matching entry point.  PyTorch supplies device memory and streams only.
A decode step's calls (``matvec``, ``moe_matvec``, ``cache_write``,
``cache_read``, ``cache_attention``) and those of a layer over many tokens
(``moe_topk``, ``gemm``, ``moe_gemm``, ``moe_combine``) pick the entry point by
their tensors' type.

A call on ``stream`` does not wait for the current one: let it wait before its
inputs are used, and the current one before its outputs are.  What such a call
allocates is memory of ``stream``.

There is no CPU path: importing this package fails when the library has not
been built (``python mxfp4_block_quantization_gb300/_build.py``), and every
call rejects tensors that are not on a CUDA device.

Method sources (vLLM pull-request summary pages): PR #43557 "Fix the E8M0
scale computation in the MXFP4 MoE CUTLASS kernel" (scale rule, tiled scale
layout, experts quant); PR #51038 "[Bugfix][Quantization] Fix MXFP4
conversion for FlashInfer CUTLASS" ([w1; w3] -> [w3; w1] swap, BF16 bias);
PR #46915 "Fix the SM90 MXFP4 MoE test weight/scale interleave" (FP4 -> BF16
table read back).
"""
import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

__all__ = [
    "MXFP4Error", "LIB_PATH", "mxfp4_scale_bytes", "mxfp4_grouped_scale_bytes_bound",
    "mxfp4_quantize", "mxfp4_quantize_grouped", "mxfp4_dequantize", "mxfp4_swap_w13",
    "mxfp4_status_string", "mxfp4_version", "quantize", "quantize_grouped", "dequantize",
    "swap_w13", "MXFP4_OK", "MXFP4_EINVAL", "MXFP4_EALIGN", "MXFP4_ESHAPE", "MXFP4_EALIAS",
    "MXFP4_ECUDA", "MXFP4_EOFFSETS", "MXFP4_EINDEX", "mxfp4_quantize_grouped_gather",
    "quantize_grouped_gather", "mxfp4_quantize_grouped_scatter", "quantize_grouped_scatter",
    "mxfp4_scatter_workspace_bytes", "mxfp4_quantize_grouped_scatter_ws",
    "mxfp4_quantize_grouped_scatter_ws_f16",
    "MXFP4_SCATTER_MAX_TOP_K", "mxfp4_quantize_f16", "mxfp4_quantize_grouped_f16",
    "mxfp4_quantize_grouped_gather_f16", "mxfp4_quantize_grouped_scatter_f16",
    "mxfp4_gather_workspace_bytes", "mxfp4_quantize_grouped_gather_ws",
    "mxfp4_quantize_grouped_gather_ws_f16", "mxfp4_quantize_grouped_gather_noalloc",
    "MXFP4_ESCRATCH", "MXFP4_NOALLOC_SCRATCH_BYTES", "mxfp4_nvfp4_scale_bytes",
    "mxfp4_quantize_nvfp4", "mxfp4_dequantize_nvfp4", "quantize_nvfp4", "dequantize_nvfp4",
    "mxfp4_nvfp4_grouped_scale_bytes_bound", "mxfp4_quantize_nvfp4_grouped",
    "quantize_nvfp4_grouped", "mxfp4_quantize_nvfp4_f16", "mxfp4_quantize_nvfp4_grouped_f16",
    "mxfp4_quantize_nvfp4_grouped_scatter", "mxfp4_quantize_nvfp4_grouped_scatter_f16",
    "quantize_nvfp4_grouped_scatter", "mxfp4_nvfp4_scatter_workspace_bytes",
    "mxfp4_quantize_nvfp4_grouped_scatter_ws", "mxfp4_quantize_nvfp4_grouped_scatter_ws_f16",
    "MXFP4_ROUTE_MAX_EXPERTS", "mxfp4_route_workspace_bytes", "mxfp4_moe_route", "moe_route",
    "MXFP4_ATTENTION_MAX_HEAD_DIM", "mxfp4_matvec", "mxfp4_matvec_nvfp4", "mxfp4_moe_matvec",
    "mxfp4_moe_matvec_nvfp4", "matvec", "matvec_nvfp4", "moe_matvec", "moe_matvec_nvfp4",
    "KVCache", "cache_alloc", "mxfp4_cache_write", "mxfp4_cache_read", "cache_write",
    "cache_read", "mxfp4_cache_attention_workspace_bytes", "mxfp4_cache_attention",
    "cache_attention", "MXFP4_TOPK_MAX", "mxfp4_moe_topk", "moe_topk", "mxfp4_gemm",
    "mxfp4_gemm_nvfp4", "gemm", "gemm_nvfp4", "mxfp4_moe_gemm", "mxfp4_moe_gemm_nvfp4",
    "moe_gemm", "moe_gemm_nvfp4", "mxfp4_moe_combine", "moe_combine",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4_gb300.so")
# The bounds-checking build (same results; every global access checked and
# counted when out of range); see _load() and mxfp4_debug_bounds_violations.
DEBUG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4_gb300_debug.so")

MXFP4_SCATTER_MAX_TOP_K = 32
MXFP4_ROUTE_MAX_EXPERTS = 8192
MXFP4_NOALLOC_SCRATCH_BYTES = 4 << 20
MXFP4_ATTENTION_MAX_HEAD_DIM = 256
MXFP4_TOPK_MAX = 32
MXFP4_OK = 0
MXFP4_EINVAL = -1
MXFP4_EALIGN = -2
MXFP4_ESHAPE = -3
MXFP4_EALIAS = -4
MXFP4_ECUDA = -5
MXFP4_EOFFSETS = -6
MXFP4_EINDEX = -7
MXFP4_ESCRATCH = -8


class MXFP4Error(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {mxfp4_status_string(code)} ({code})")


def _load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python mxfp4_block_quantization_gb300/_build.py` (nvcc, sm_103a)")
    L = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.mxfp4_scale_bytes.restype = ctypes.c_size_t
    L.mxfp4_scale_bytes.argtypes = [i64, i64]
    L.mxfp4_grouped_scale_bytes_bound.restype = ctypes.c_size_t
    L.mxfp4_grouped_scale_bytes_bound.argtypes = [i64, i32, i64]
    L.mxfp4_quantize.restype = ctypes.c_int
    L.mxfp4_quantize.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    L.mxfp4_quantize_f16.restype = ctypes.c_int
    L.mxfp4_quantize_f16.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    L.mxfp4_quantize_grouped.restype = ctypes.c_int
    L.mxfp4_quantize_grouped.argtypes = [vp, i64, i64, vp, i32, vp, vp, vp, vp, vp]
    L.mxfp4_quantize_grouped_f16.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_f16.argtypes = [vp, i64, i64, vp, i32, vp, vp, vp, vp, vp]
    L.mxfp4_quantize_grouped_gather_f16.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_gather_f16.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, vp, vp,
                                                    vp, vp, vp]
    L.mxfp4_quantize_grouped_scatter_f16.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_scatter_f16.argtypes = [vp, i64, i64, i64, vp, i32, i64, vp, i32,
                                                     vp, vp, vp, vp, vp]
    L.mxfp4_gather_workspace_bytes.restype = ctypes.c_size_t
    L.mxfp4_gather_workspace_bytes.argtypes = [i64, i64, i32, i64]
    for name in ("mxfp4_quantize_grouped_gather_ws", "mxfp4_quantize_grouped_gather_ws_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, vp, ctypes.c_size_t,
                                     vp, vp, vp, vp, vp]
    L.mxfp4_quantize_grouped_gather_noalloc.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_gather_noalloc.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, vp,
                                                        vp, vp, vp, vp]
    L.mxfp4_quantize_grouped_gather.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_gather.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, vp, vp, vp,
                                                vp, vp]
    L.mxfp4_quantize_grouped_scatter.restype = ctypes.c_int
    L.mxfp4_quantize_grouped_scatter.argtypes = [vp, i64, i64, i64, vp, i32, i64, vp, i32, vp,
                                                 vp, vp, vp, vp]
    L.mxfp4_scatter_workspace_bytes.restype = ctypes.c_size_t
    L.mxfp4_scatter_workspace_bytes.argtypes = [i64, i64, i32, i64]
    for name in ("mxfp4_quantize_grouped_scatter_ws", "mxfp4_quantize_grouped_scatter_ws_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, i64, vp, i32, i64, vp, i32, vp,
                                     ctypes.c_size_t, vp, vp, vp, vp, vp]
    L.mxfp4_dequantize.restype = ctypes.c_int
    L.mxfp4_dequantize.argtypes = [vp, vp, i64, i64, vp, vp]
    L.mxfp4_swap_w13.restype = ctypes.c_int
    L.mxfp4_swap_w13.argtypes = [vp, vp, vp, i32, i64, i64, i32, vp, vp, vp, vp, i64, vp, vp]
    L.mxfp4_nvfp4_scale_bytes.restype = ctypes.c_size_t
    L.mxfp4_nvfp4_scale_bytes.argtypes = [i64, i64]
    for name in ("mxfp4_quantize_nvfp4", "mxfp4_quantize_nvfp4_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
    L.mxfp4_nvfp4_grouped_scale_bytes_bound.restype = ctypes.c_size_t
    L.mxfp4_nvfp4_grouped_scale_bytes_bound.argtypes = [i64, i32, i64]
    for name in ("mxfp4_quantize_nvfp4_grouped", "mxfp4_quantize_nvfp4_grouped_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp]
    for name in ("mxfp4_quantize_nvfp4_grouped_scatter",
                 "mxfp4_quantize_nvfp4_grouped_scatter_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, i64, vp, i32, i64, vp, i32, vp, vp, vp, vp, vp,
                                     vp]
    for name in ("mxfp4_quantize_nvfp4_grouped_scatter_ws",
                 "mxfp4_quantize_nvfp4_grouped_scatter_ws_f16"):
        getattr(L, name).restype = ctypes.c_int
        getattr(L, name).argtypes = [vp, i64, i64, i64, vp, i32, i64, vp, i32, vp, vp,
                                     ctypes.c_size_t, vp, vp, vp, vp, vp]
    L.mxfp4_nvfp4_scatter_workspace_bytes.restype = ctypes.c_size_t
    L.mxfp4_nvfp4_scatter_workspace_bytes.argtypes = [i64, i32, i64]
    L.mxfp4_dequantize_nvfp4.restype = ctypes.c_int
    L.mxfp4_dequantize_nvfp4.argtypes = [vp, vp, vp, i64, i64, vp, vp]
    L.mxfp4_route_workspace_bytes.restype = ctypes.c_size_t
    L.mxfp4_route_workspace_bytes.argtypes = [i64, i32, i32]
    L.mxfp4_moe_route.restype = ctypes.c_int
    L.mxfp4_moe_route.argtypes = [vp, i64, i32, i32, vp, ctypes.c_size_t, vp, vp, vp, vp, vp]
    f32, size = ctypes.c_float, ctypes.c_size_t
    decode = L.decode = {}  # (call, NVFP4, FP16) -> entry point and its name
    for nv in (False, True):
        for f16 in (False, True):
            tail = ("_nvfp4" if nv else "") + ("_f16" if f16 else "")
            g1, g2 = ([vp], [vp, vp]) if nv else ([], [])
            for name, args in (
                    ("matvec", [vp, i64, i64, i64, vp, vp] + g1 + [i64, vp, i64, i32, vp]),
                    ("moe_matvec", [vp, i64, i64, i64, vp, i64, vp, i32, vp, vp] + g1 +
                     [i64, vp, i64, i32, vp, vp]),
                    ("cache_write", [vp, vp, i64, i32, i32, i64, i64, i64, i64, vp, i64, i32] +
                     g2 + [vp, vp, vp, vp, vp, vp]),
                    ("cache_read", [vp, vp, vp, vp] + g2 + [i64, i32, i32, i32, vp, i64, vp, vp,
                                                            vp, vp]),
                    ("cache_attention", [vp, i64, i32, i32, i64, i64, vp, vp, vp, vp] + g2 +
                     [i64, i32, i32, vp, i64, i64, vp, f32, i32, vp, size, vp, vp, vp, vp])):
                fn = getattr(L, "mxfp4_" + name + tail)
                fn.restype = ctypes.c_int
                fn.argtypes = args
                decode[name, nv, f16] = fn, "mxfp4_" + name + tail
    layer = L.layer = {}  # (call, type) or (call, NVFP4, FP16) -> entry point and its name
    for tail, kind in (("", torch.bfloat16), ("_f16", torch.float16), ("_f32", torch.float32)):
        fn = getattr(L, "mxfp4_moe_topk" + tail)
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, i64, i32, i64, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, vp]
        layer["moe_topk", kind] = fn, "mxfp4_moe_topk" + tail
    for nv in (False, True):
        for f16 in (False, True):
            tail = ("_nvfp4" if nv else "") + ("_f16" if f16 else "")
            g = [vp] if nv else []
            for name, args in (
                    ("gemm", [vp, vp] + g + [i64, i64, vp, vp] + g +
                     [i64, vp, i32, i32, vp, i64, vp, i64, vp]),
                    ("moe_gemm", [vp, vp] + g + [i64, i64, vp, i32, vp, vp] + g +
                     [i64, vp, i32, i32, vp, i64, vp, vp])):
                fn = getattr(L, "mxfp4_" + name + tail)
                fn.restype = ctypes.c_int
                fn.argtypes = args
                layer[name, nv, f16] = fn, "mxfp4_" + name + tail
    for f16, tail in ((False, ""), (True, "_f16")):
        fn = getattr(L, "mxfp4_moe_combine" + tail)
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, i32, vp, i64, vp, i64, vp, vp]
        layer["moe_combine", f16] = fn, "mxfp4_moe_combine" + tail
    L.mxfp4_cache_attention_workspace_bytes.restype = size
    L.mxfp4_cache_attention_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i64]
    L.mxfp4_status_string.restype = ctypes.c_char_p
    L.mxfp4_status_string.argtypes = [ctypes.c_int]
    L.mxfp4_version.restype = ctypes.c_int
    L.mxfp4_version.argtypes = []
    if hasattr(L, "mxfp4_debug_bounds_violations"):
        L.mxfp4_debug_bounds_violations.restype = ctypes.c_int64
        L.mxfp4_debug_bounds_violations.argtypes = []
        L.mxfp4_debug_stall_products.restype = ctypes.c_int
        L.mxfp4_debug_stall_products.argtypes = [i32]
    return L


_lib = _load()


# ------------------------------------------------------------------ helpers
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's raw handle without building a torch Stream object (a
# measurable share of a call's host time); the public path where torch lacks it.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_current_stream is not None:
        return ctypes.c_void_p(_raw_current_stream(device.index))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(name, t, dtype=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _need_bytes(name, t, nbytes):
    """``t`` (if given) must be contiguous and hold at least ``nbytes`` bytes:
    the library sees only its pointer and reads or writes the whole extent
    the call's sizes imply, so a short or strided buffer is refused here,
    before anything is launched.  ``nbytes`` <= 0 (sizes the library itself
    rejects) checks contiguity only."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes; this call needs {nbytes}")


def _check(rc, where):
    if rc != MXFP4_OK:
        raise MXFP4Error(rc, where)


def _device_of(*tensors):
    """The one CUDA device all given tensors live on (the library launches on
    the current device, so every call switches to it)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            devs = sorted({str(u.device) for u in tensors if u is not None})
            raise ValueError(f"all tensors must be on the same CUDA device, got {devs}")
    if dev is None:
        raise ValueError("no tensor given")
    return dev


def _switch(device):
    """The library launches on the current device: make ``device`` current for
    the call, or do nothing when it already is (the usual case, and a
    measurable share of a call's host time)."""
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


# ------------------------------------------------------- C entry points
@functools.lru_cache(maxsize=1024)
def mxfp4_scale_bytes(M: int, K: int) -> int:
    return int(_lib.mxfp4_scale_bytes(int(M), int(K)))


@functools.lru_cache(maxsize=1024)
def mxfp4_grouped_scale_bytes_bound(total_rows: int, E: int, K: int) -> int:
    return int(_lib.mxfp4_grouped_scale_bytes_bound(int(total_rows), int(E), int(K)))


def mxfp4_status_string(code: int) -> str:
    return _lib.mxfp4_status_string(int(code)).decode()


def mxfp4_version() -> int:
    return int(_lib.mxfp4_version())


def mxfp4_quantize(x, codes, scales, stream=None) -> None:
    """BF16 ``x`` [M, K] (row stride may exceed K) -> ``codes`` uint8 [M, K/2]
    and ``scales`` uint8 [mxfp4_scale_bytes(M, K)] (128x4 tiled)."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    _need_bytes("codes", codes, M * (K // 2))
    _need_bytes("scales", scales, mxfp4_scale_bytes(M, K))
    with _switch(_device_of(x, codes, scales)):
        _check(_lib.mxfp4_quantize(_ptr(x), M, K, x.stride(0), _ptr(codes), _ptr(scales),
                                   _stream(stream, x.device)), "mxfp4_quantize")


def mxfp4_quantize_f16(x, codes, scales, stream=None) -> None:
    """FP16 ``x`` [M, K] (row stride may exceed K) -> the same codes and tiled
    scales as mxfp4_quantize produces for BF16 input."""
    _need_cuda("x", x, torch.float16)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    _need_bytes("codes", codes, M * (K // 2))
    _need_bytes("scales", scales, mxfp4_scale_bytes(M, K))
    with _switch(_device_of(x, codes, scales)):
        _check(_lib.mxfp4_quantize_f16(_ptr(x), M, K, x.stride(0), _ptr(codes), _ptr(scales),
                                       _stream(stream, x.device)), "mxfp4_quantize_f16")


def _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status, rows, K,
                          scale_bound):
    """The buffers of a grouped call over ``rows`` expert-sorted rows."""
    E = expert_offsets.numel() - 1
    _need_bytes("expert_offsets", expert_offsets, 4 * (E + 1))
    _need_bytes("codes", codes, rows * (K // 2))
    _need_bytes("scales", scales, scale_bound(rows, E, K) if E >= 0 and rows >= 0 else 0)
    _need_bytes("scale_row_offsets", scale_row_offsets, 4 * (E + 1))
    _need_bytes("status", status, 4)


def _grouped(x, expert_offsets, codes, scales, scale_row_offsets, status, stream, f16):
    name = "mxfp4_quantize_grouped" + ("_f16" if f16 else "")
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor")
    total, K = x.shape
    E = expert_offsets.numel() - 1
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status, total, K,
                          mxfp4_grouped_scale_bytes_bound)
    with _switch(_device_of(x, expert_offsets, codes, scales, scale_row_offsets, status)):
        _check(getattr(_lib, name)(_ptr(x), total, K, _ptr(expert_offsets), E, _ptr(codes),
                                   _ptr(scales), _ptr(scale_row_offsets), _ptr(status),
                                   _stream(stream, x.device)), name)


def mxfp4_quantize_grouped(x, expert_offsets, codes, scales, scale_row_offsets, status=None,
                           stream=None) -> None:
    """Per-expert quantize of contiguous BF16 rows ``x`` [total_rows, K]
    delimited by int32 ``expert_offsets`` [E+1] (device)."""
    _grouped(x, expert_offsets, codes, scales, scale_row_offsets, status, stream, False)


def mxfp4_quantize_grouped_f16(x, expert_offsets, codes, scales, scale_row_offsets, status=None,
                               stream=None) -> None:
    """mxfp4_quantize_grouped for FP16 ``x``."""
    _grouped(x, expert_offsets, codes, scales, scale_row_offsets, status, stream, True)


def _gather(x, row_index, expert_offsets, codes, scales, scale_row_offsets, status, stream, f16):
    name = "mxfp4_quantize_grouped_gather" + ("_f16" if f16 else "")
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("row_index", row_index, torch.int32)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if not row_index.is_contiguous():
        raise ValueError("row_index must be contiguous")
    n_src, K = x.shape
    E = expert_offsets.numel() - 1
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status,
                          row_index.numel(), K, mxfp4_grouped_scale_bytes_bound)
    with _switch(_device_of(x, row_index, expert_offsets, codes, scales,
                                      scale_row_offsets, status)):
        _check(getattr(_lib, name)(
            _ptr(x), n_src, K, x.stride(0), _ptr(row_index), row_index.numel(),
            _ptr(expert_offsets), E, _ptr(codes), _ptr(scales), _ptr(scale_row_offsets),
            _ptr(status), _stream(stream, x.device)), name)


def mxfp4_quantize_grouped_gather(x, row_index, expert_offsets, codes, scales, scale_row_offsets,
                                  status=None, stream=None) -> None:
    """Grouped quantize of the rows ``x[row_index]`` (int32 device indices)
    without materialising the gathered BF16 matrix."""
    _gather(x, row_index, expert_offsets, codes, scales, scale_row_offsets, status, stream, False)


def mxfp4_quantize_grouped_gather_f16(x, row_index, expert_offsets, codes, scales,
                                      scale_row_offsets, status=None, stream=None) -> None:
    """mxfp4_quantize_grouped_gather for FP16 ``x``."""
    _gather(x, row_index, expert_offsets, codes, scales, scale_row_offsets, status, stream, True)


@functools.lru_cache(maxsize=1024)
def mxfp4_gather_workspace_bytes(num_src_rows: int, total_rows: int, E: int, K: int) -> int:
    return int(_lib.mxfp4_gather_workspace_bytes(int(num_src_rows), int(total_rows), int(E),
                                                 int(K)))


def _gather_ws(x, row_index, expert_offsets, workspace, codes, scales, scale_row_offsets, status,
               stream, f16):
    name = "mxfp4_quantize_grouped_gather_ws" + ("_f16" if f16 else "")
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("row_index", row_index, torch.int32)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("workspace", workspace)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if not row_index.is_contiguous() or not workspace.is_contiguous():
        raise ValueError("row_index and workspace must be contiguous")
    n_src, K = x.shape
    E = expert_offsets.numel() - 1
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status,
                          row_index.numel(), K, mxfp4_grouped_scale_bytes_bound)
    with _switch(_device_of(x, row_index, expert_offsets, workspace, codes, scales,
                                      scale_row_offsets, status)):
        _check(getattr(_lib, name)(
            _ptr(x), n_src, K, x.stride(0), _ptr(row_index), row_index.numel(),
            _ptr(expert_offsets), E, _ptr(workspace), workspace.numel() * workspace.element_size(),
            _ptr(codes), _ptr(scales), _ptr(scale_row_offsets), _ptr(status),
            _stream(stream, x.device)), name)


def mxfp4_quantize_grouped_gather_ws(x, row_index, expert_offsets, workspace, codes, scales,
                                     scale_row_offsets, status=None, stream=None) -> None:
    """mxfp4_quantize_grouped_gather through the scatter path: the inverse
    map is built in ``workspace`` (device, >= mxfp4_gather_workspace_bytes)."""
    _gather_ws(x, row_index, expert_offsets, workspace, codes, scales, scale_row_offsets, status,
               stream, False)


def mxfp4_quantize_grouped_gather_noalloc(x, row_index, expert_offsets, codes, scales,
                                          scale_row_offsets, status=None, stream=None) -> None:
    """mxfp4_quantize_grouped_gather_ws with the library's fixed scratch
    buffer (no workspace, no allocation); calls must not overlap on the GPU."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("row_index", row_index, torch.int32)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if not row_index.is_contiguous():
        raise ValueError("row_index must be contiguous")
    n_src, K = x.shape
    E = expert_offsets.numel() - 1
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status,
                          row_index.numel(), K, mxfp4_grouped_scale_bytes_bound)
    with _switch(_device_of(x, row_index, expert_offsets, codes, scales,
                                      scale_row_offsets, status)):
        _check(_lib.mxfp4_quantize_grouped_gather_noalloc(
            _ptr(x), n_src, K, x.stride(0), _ptr(row_index), row_index.numel(),
            _ptr(expert_offsets), E, _ptr(codes), _ptr(scales), _ptr(scale_row_offsets),
            _ptr(status), _stream(stream, x.device)), "mxfp4_quantize_grouped_gather_noalloc")


def mxfp4_quantize_grouped_gather_ws_f16(x, row_index, expert_offsets, workspace, codes, scales,
                                         scale_row_offsets, status=None, stream=None) -> None:
    """mxfp4_quantize_grouped_gather_ws for FP16 ``x``."""
    _gather_ws(x, row_index, expert_offsets, workspace, codes, scales, scale_row_offsets, status,
               stream, True)


def _scatter(x, dest_rows, expert_offsets, total_rows, codes, scales, scale_row_offsets, status,
             stream, f16, workspace=None):
    name = ("mxfp4_quantize_grouped_scatter" + ("_ws" if workspace is not None else "") +
            ("_f16" if f16 else ""))
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("workspace", workspace, torch.uint8)
    _need_cuda("dest_rows", dest_rows, torch.int32)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if dest_rows.dim() != 2 or dest_rows.shape[0] != x.shape[0] or not dest_rows.is_contiguous():
        raise ValueError("dest_rows must be a contiguous [num_tokens, top_k] tensor")
    T, K = x.shape
    E = expert_offsets.numel() - 1
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status,
                          int(total_rows), K, mxfp4_grouped_scale_bytes_bound)
    _need_bytes("workspace", workspace, 0)
    ws = () if workspace is None else (_ptr(workspace), workspace.numel())
    with _switch(_device_of(x, dest_rows, expert_offsets, codes, scales,
                                      scale_row_offsets, status, workspace)):
        _check(getattr(_lib, name)(
            _ptr(x), T, K, x.stride(0), _ptr(dest_rows), dest_rows.shape[1], int(total_rows),
            _ptr(expert_offsets), E, *ws, _ptr(codes), _ptr(scales), _ptr(scale_row_offsets),
            _ptr(status), _stream(stream, x.device)), name)


def mxfp4_quantize_grouped_scatter(x, dest_rows, expert_offsets, total_rows: int, codes, scales,
                                   scale_row_offsets, status=None, stream=None) -> None:
    """Grouped quantize with the dispatch given token -> rows: route j of
    token t is row ``dest_rows[t, j]`` (int32 device [T, top_k], -1 = not
    dispatched) of the ``total_rows``-row expert-sorted batch.  Each token
    row is read and quantized once; rows no route targets are not written."""
    _scatter(x, dest_rows, expert_offsets, total_rows, codes, scales, scale_row_offsets, status,
             stream, False)


def mxfp4_quantize_grouped_scatter_f16(x, dest_rows, expert_offsets, total_rows: int, codes,
                                       scales, scale_row_offsets, status=None,
                                       stream=None) -> None:
    """mxfp4_quantize_grouped_scatter for FP16 ``x``."""
    _scatter(x, dest_rows, expert_offsets, total_rows, codes, scales, scale_row_offsets, status,
             stream, True)


@functools.lru_cache(maxsize=1024)
def mxfp4_scatter_workspace_bytes(num_tokens: int, total_rows: int, E: int, K: int) -> int:
    return int(_lib.mxfp4_scatter_workspace_bytes(int(num_tokens), int(total_rows), int(E),
                                                  int(K)))


def mxfp4_quantize_grouped_scatter_ws(x, dest_rows, expert_offsets, total_rows: int, workspace,
                                      codes, scales, scale_row_offsets, status=None,
                                      stream=None) -> None:
    """mxfp4_quantize_grouped_scatter with identical results, staging each
    token's scale words once in ``workspace`` (uint8 device, >=
    mxfp4_scatter_workspace_bytes) and writing the tiled scales whole."""
    _scatter(x, dest_rows, expert_offsets, total_rows, codes, scales, scale_row_offsets, status,
             stream, False, workspace)


def mxfp4_quantize_grouped_scatter_ws_f16(x, dest_rows, expert_offsets, total_rows: int,
                                          workspace, codes, scales, scale_row_offsets,
                                          status=None, stream=None) -> None:
    """mxfp4_quantize_grouped_scatter_ws for FP16 ``x``."""
    _scatter(x, dest_rows, expert_offsets, total_rows, codes, scales, scale_row_offsets, status,
             stream, True, workspace)


@functools.lru_cache(maxsize=1024)
def mxfp4_route_workspace_bytes(num_tokens: int, top_k: int, E: int) -> int:
    return int(_lib.mxfp4_route_workspace_bytes(int(num_tokens), int(top_k), int(E)))


def mxfp4_moe_route(topk_ids, num_experts: int, workspace, expert_offsets, dest_rows,
                    row_index=None, status=None, stream=None) -> None:
    """The dispatch permutation from the router's expert ids ``topk_ids``
    [num_tokens, top_k] (int32, -1: not dispatched): ``expert_offsets``
    [E+1], ``dest_rows`` [num_tokens, top_k] and, if given, ``row_index``
    [num_tokens * top_k] (the token of every row), in order of expert, then
    of entry.  ``workspace``: >= mxfp4_route_workspace_bytes bytes."""
    for name, t in (("topk_ids", topk_ids), ("expert_offsets", expert_offsets),
                    ("dest_rows", dest_rows), ("row_index", row_index), ("status", status)):
        _need_cuda(name, t, torch.int32)
    _need_cuda("workspace", workspace)
    for name, t in (("topk_ids", topk_ids), ("dest_rows", dest_rows)):
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [num_tokens, top_k] tensor")
    if dest_rows.shape != topk_ids.shape:
        raise ValueError("dest_rows must have the shape of topk_ids")
    T, top_k = topk_ids.shape
    _need_bytes("workspace", workspace, 0)
    _need_bytes("expert_offsets", expert_offsets, 4 * (int(num_experts) + 1))
    _need_bytes("row_index", row_index, 4 * T * top_k)
    _need_bytes("status", status, 4)
    with _switch(_device_of(topk_ids, workspace, expert_offsets, dest_rows,
                                      row_index, status)):
        _check(_lib.mxfp4_moe_route(_ptr(topk_ids), T, top_k, int(num_experts), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _ptr(expert_offsets), _ptr(dest_rows), _ptr(row_index),
                                    _ptr(status), _stream(stream, topk_ids.device)),
               "mxfp4_moe_route")


def mxfp4_dequantize(codes, scales, M: int, K: int, y, stream=None) -> None:
    """``codes`` [M, K/2] + tiled ``scales`` -> BF16 ``y`` [M, K] (contiguous)."""
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("y", y, torch.bfloat16)
    M, K = int(M), int(K)
    _need_bytes("codes", codes, M * (K // 2))
    _need_bytes("scales", scales, mxfp4_scale_bytes(M, K))
    _need_bytes("y", y, 2 * M * K)
    with _switch(_device_of(codes, scales, y)):
        _check(_lib.mxfp4_dequantize(_ptr(codes), _ptr(scales), int(M), int(K), _ptr(y),
                                     _stream(stream, y.device)), "mxfp4_dequantize")


def mxfp4_swap_w13(codes_in, scales_in, w13_bias_in, E: int, two_n: int, K: int,
                   scales_tiled: int, codes_out, scales_out, w13_bias_out=None,
                   w2_bias_in=None, w2_bias_out=None, stream=None) -> None:
    """[w1; w3] -> [w3; w1] of codes, scales (flat or tiled per expert) and
    FP32 biases (cast to BF16); the w2 bias is cast only."""
    for n, t, d in (("codes_in", codes_in, torch.uint8), ("scales_in", scales_in, torch.uint8),
                    ("codes_out", codes_out, torch.uint8), ("scales_out", scales_out, torch.uint8),
                    ("w13_bias_in", w13_bias_in, torch.float32),
                    ("w13_bias_out", w13_bias_out, torch.bfloat16),
                    ("w2_bias_in", w2_bias_in, torch.float32),
                    ("w2_bias_out", w2_bias_out, torch.bfloat16)):
        _need_cuda(n, t, d)
    dev = _device_of(codes_in, scales_in, codes_out, scales_out, w13_bias_in, w13_bias_out,
                     w2_bias_in, w2_bias_out)
    n2 = w2_bias_in.numel() if w2_bias_in is not None else 0
    E, two_n, K = int(E), int(two_n), int(K)
    code_bytes = E * two_n * (K // 2)
    scale_bytes = (E * mxfp4_scale_bytes(two_n, K) if scales_tiled else E * two_n * (K // 32))
    _need_bytes("codes_in", codes_in, code_bytes)
    _need_bytes("codes_out", codes_out, code_bytes)
    _need_bytes("scales_in", scales_in, scale_bytes)
    _need_bytes("scales_out", scales_out, scale_bytes)
    _need_bytes("w13_bias_in", w13_bias_in, 4 * E * two_n)
    if w13_bias_in is not None:
        _need_bytes("w13_bias_out", w13_bias_out, 2 * E * two_n)
    _need_bytes("w2_bias_in", w2_bias_in, 4 * n2)
    if w2_bias_in is not None:
        _need_bytes("w2_bias_out", w2_bias_out, 2 * n2)
    with _switch(dev):
        _check(_lib.mxfp4_swap_w13(_ptr(codes_in), _ptr(scales_in), _ptr(w13_bias_in), int(E),
                                   int(two_n), int(K), int(scales_tiled), _ptr(codes_out),
                                   _ptr(scales_out), _ptr(w13_bias_out), _ptr(w2_bias_in), n2,
                                   _ptr(w2_bias_out), _stream(stream, dev)), "mxfp4_swap_w13")


@functools.lru_cache(maxsize=1024)
def mxfp4_nvfp4_scale_bytes(M: int, K: int) -> int:
    return int(_lib.mxfp4_nvfp4_scale_bytes(int(M), int(K)))


def _nvfp4(x, global_scale, codes, scales, stream, f16) -> None:
    name = "mxfp4_quantize_nvfp4" + ("_f16" if f16 else "")
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("global_scale", global_scale, torch.float32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    _need_bytes("global_scale", global_scale, 4)
    _need_bytes("codes", codes, M * (K // 2))
    _need_bytes("scales", scales, mxfp4_nvfp4_scale_bytes(M, K))
    with _switch(_device_of(x, global_scale, codes, scales)):
        _check(getattr(_lib, name)(_ptr(x), M, K, x.stride(0), _ptr(global_scale), _ptr(codes),
                                   _ptr(scales), _stream(stream, x.device)), name)


def mxfp4_quantize_nvfp4(x, global_scale, codes, scales, stream=None) -> None:
    """NVFP4: BF16 ``x`` [M, K] with float32 ``global_scale`` (1 element,
    device) -> codes [M, K/2] + tiled E4M3 scales."""
    _nvfp4(x, global_scale, codes, scales, stream, False)


def mxfp4_quantize_nvfp4_f16(x, global_scale, codes, scales, stream=None) -> None:
    """NVFP4 of FP16 ``x``; everything else as mxfp4_quantize_nvfp4."""
    _nvfp4(x, global_scale, codes, scales, stream, True)


@functools.lru_cache(maxsize=1024)
def mxfp4_nvfp4_grouped_scale_bytes_bound(total_rows: int, E: int, K: int) -> int:
    return int(_lib.mxfp4_nvfp4_grouped_scale_bytes_bound(int(total_rows), int(E), int(K)))


def _nvfp4_grouped(x, expert_offsets, global_scales, codes, scales, scale_row_offsets, status,
                   stream, f16) -> None:
    name = "mxfp4_quantize_nvfp4_grouped" + ("_f16" if f16 else "")
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("global_scales", global_scales, torch.float32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D tensor")
    total, K = x.shape
    E = expert_offsets.numel() - 1
    if global_scales.numel() != E:
        raise ValueError("global_scales needs one entry per expert")
    _need_bytes("global_scales", global_scales, 4 * E)
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status, total, K,
                          mxfp4_nvfp4_grouped_scale_bytes_bound)
    with _switch(_device_of(x, expert_offsets, global_scales, codes, scales,
                                      scale_row_offsets, status)):
        _check(getattr(_lib, name)(
            _ptr(x), total, K, _ptr(expert_offsets), E, _ptr(global_scales), _ptr(codes),
            _ptr(scales), _ptr(scale_row_offsets), _ptr(status), _stream(stream, x.device)), name)


def mxfp4_quantize_nvfp4_grouped(x, expert_offsets, global_scales, codes, scales,
                                 scale_row_offsets, status=None, stream=None) -> None:
    """NVFP4 experts quant: segment e of the contiguous BF16 ``x`` with global
    scale ``global_scales[e]`` (float32 device [E])."""
    _nvfp4_grouped(x, expert_offsets, global_scales, codes, scales, scale_row_offsets, status,
                   stream, False)


def mxfp4_quantize_nvfp4_grouped_f16(x, expert_offsets, global_scales, codes, scales,
                                     scale_row_offsets, status=None, stream=None) -> None:
    """NVFP4 experts quant of FP16 ``x``; everything else as the BF16 form."""
    _nvfp4_grouped(x, expert_offsets, global_scales, codes, scales, scale_row_offsets, status,
                   stream, True)


def _nvfp4_scatter(x, dest_rows, expert_offsets, total_rows, global_scales, codes, scales,
                   scale_row_offsets, status, stream, f16, workspace=None) -> None:
    name = ("mxfp4_quantize_nvfp4_grouped_scatter" + ("_ws" if workspace is not None else "") +
            ("_f16" if f16 else ""))
    _need_cuda("x", x, torch.float16 if f16 else torch.bfloat16)
    _need_cuda("workspace", workspace, torch.uint8)
    _need_cuda("dest_rows", dest_rows, torch.int32)
    _need_cuda("expert_offsets", expert_offsets, torch.int32)
    _need_cuda("global_scales", global_scales, torch.float32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("scale_row_offsets", scale_row_offsets, torch.int32)
    _need_cuda("status", status, torch.int32)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if dest_rows.dim() != 2 or dest_rows.shape[0] != x.shape[0] or not dest_rows.is_contiguous():
        raise ValueError("dest_rows must be a contiguous [num_tokens, top_k] tensor")
    T, K = x.shape
    E = expert_offsets.numel() - 1
    if global_scales.numel() != E:
        raise ValueError("global_scales needs one entry per expert")
    _need_bytes("global_scales", global_scales, 4 * E)
    _need_grouped_outputs(expert_offsets, codes, scales, scale_row_offsets, status,
                          int(total_rows), K, mxfp4_nvfp4_grouped_scale_bytes_bound)
    _need_bytes("workspace", workspace, 0)
    ws = () if workspace is None else (_ptr(workspace), workspace.numel())
    with _switch(_device_of(x, dest_rows, expert_offsets, global_scales, codes, scales,
                                      scale_row_offsets, status, workspace)):
        _check(getattr(_lib, name)(
            _ptr(x), T, K, x.stride(0), _ptr(dest_rows), dest_rows.shape[1], int(total_rows),
            _ptr(expert_offsets), E, _ptr(global_scales), *ws, _ptr(codes), _ptr(scales),
            _ptr(scale_row_offsets), _ptr(status), _stream(stream, x.device)), name)


def mxfp4_quantize_nvfp4_grouped_scatter(x, dest_rows, expert_offsets, total_rows: int,
                                         global_scales, codes, scales, scale_row_offsets,
                                         status=None, stream=None) -> None:
    """NVFP4 experts quant with the dispatch as a scatter: route j of token t
    is row ``dest_rows[t, j]`` (-1 = not dispatched); segment e uses
    ``global_scales[e]``.  Rows no route targets are not written."""
    _nvfp4_scatter(x, dest_rows, expert_offsets, total_rows, global_scales, codes, scales,
                   scale_row_offsets, status, stream, False)


def mxfp4_quantize_nvfp4_grouped_scatter_f16(x, dest_rows, expert_offsets, total_rows: int,
                                             global_scales, codes, scales, scale_row_offsets,
                                             status=None, stream=None) -> None:
    """mxfp4_quantize_nvfp4_grouped_scatter for FP16 ``x``."""
    _nvfp4_scatter(x, dest_rows, expert_offsets, total_rows, global_scales, codes, scales,
                   scale_row_offsets, status, stream, True)


@functools.lru_cache(maxsize=1024)
def mxfp4_nvfp4_scatter_workspace_bytes(total_rows: int, E: int, K: int) -> int:
    return int(_lib.mxfp4_nvfp4_scatter_workspace_bytes(int(total_rows), int(E), int(K)))


def mxfp4_quantize_nvfp4_grouped_scatter_ws(x, dest_rows, expert_offsets, total_rows: int,
                                            global_scales, workspace, codes, scales,
                                            scale_row_offsets, status=None, stream=None) -> None:
    """mxfp4_quantize_nvfp4_grouped_scatter with identical results, each
    route's scale bytes staged by padded row in ``workspace`` (uint8 device, >=
    mxfp4_nvfp4_scatter_workspace_bytes) and tiled by a second kernel."""
    _nvfp4_scatter(x, dest_rows, expert_offsets, total_rows, global_scales, codes, scales,
                   scale_row_offsets, status, stream, False, workspace)


def mxfp4_quantize_nvfp4_grouped_scatter_ws_f16(x, dest_rows, expert_offsets, total_rows: int,
                                                global_scales, workspace, codes, scales,
                                                scale_row_offsets, status=None,
                                                stream=None) -> None:
    """mxfp4_quantize_nvfp4_grouped_scatter_ws for FP16 ``x``."""
    _nvfp4_scatter(x, dest_rows, expert_offsets, total_rows, global_scales, codes, scales,
                   scale_row_offsets, status, stream, True, workspace)


def mxfp4_dequantize_nvfp4(codes, scales, global_scale, M: int, K: int, y, stream=None) -> None:
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    _need_cuda("global_scale", global_scale, torch.float32)
    _need_cuda("y", y, torch.bfloat16)
    M, K = int(M), int(K)
    _need_bytes("global_scale", global_scale, 4)
    _need_bytes("codes", codes, M * (K // 2))
    _need_bytes("scales", scales, mxfp4_nvfp4_scale_bytes(M, K))
    _need_bytes("y", y, 2 * M * K)
    with _switch(_device_of(codes, scales, global_scale, y)):
        _check(_lib.mxfp4_dequantize_nvfp4(_ptr(codes), _ptr(scales), _ptr(global_scale), int(M),
                                           int(K), _ptr(y), _stream(stream, y.device)),
               "mxfp4_dequantize_nvfp4")


# ------------------------------------------- products with 4-bit weights
# These calls are made once a layer and token, so their checks read each
# tensor property once (a few us of host time per call).
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _decode_call(key, device, stream, args):
    _launch(_lib.decode[key], device, stream, args)


def _launch(entry, device, stream, args):
    """Launch an entry point on ``device`` (an index): args, then the stream."""
    fn, name = entry
    if stream is not None:
        stream = stream.cuda_stream
    elif _raw_current_stream is not None:
        stream = _raw_current_stream(device)
    else:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device == _get_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc:
        raise MXFP4Error(rc, name)


def _half_type(name, t):
    """Whether ``t`` is FP16 (True) or BF16 (False)."""
    d = t.dtype
    if d is torch.float16:
        return True
    if d is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float16, got {d}")
    return False


def _device_index(name, t):
    """The index of the CUDA device of the tensor ``t``."""
    device = t.get_device() if isinstance(t, torch.Tensor) else -1
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    return device


def _address(name, t, device, dtype, nbytes):
    """The address of ``t`` (None: no address), a contiguous ``dtype`` tensor
    on ``device`` that holds at least ``nbytes``."""
    if t is None:
        return None
    try:
        if (t.get_device() == device and (dtype is None or t.dtype is dtype) and
                t.is_contiguous() and t.numel() * t.element_size() >= nbytes):
            return t.data_ptr()
    except AttributeError:
        pass
    if _device_index(name, t) != device:  # says what is wrong
        raise ValueError(f"all tensors must be on the same CUDA device, {name} is on {t.device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes; this call needs {nbytes}")
    return t.data_ptr()


def _matrix(name, t, device, dtypes):
    """(address, rows, columns, row stride) of a 2-D tensor with unit column
    stride, of one of ``dtypes``."""
    if _device_index(name, t) != device:
        raise ValueError(f"all tensors must be on the same CUDA device, {name} is on {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    (rows, cols), (row_stride, col_stride) = t.shape, t.stride()
    if col_stride != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), rows, cols, row_stride if rows > 1 else cols


def _product(x, codes, scales, global_scales, y, E, nvfp4):
    """The checked arguments that the dense and the experts' products share:
    (FP16, device, x's, y's, the weights' [, global scales'], N)."""
    f16 = _half_type("x", x) if isinstance(x, torch.Tensor) else False
    device = _device_index("x", x)
    xa = _matrix("x", x, device, (x.dtype,))
    ya = _matrix("y", y, device, (x.dtype, torch.float32))
    K, N = xa[2], codes.shape[-2]
    if codes.shape[-1] * 2 != K:
        raise ValueError(f"codes hold {codes.shape[-1] * 2} elements per row, x has {K}")
    if ya[2] != N:
        raise ValueError(f"y must have {N} columns, got {ya[2]}")
    per = mxfp4_nvfp4_scale_bytes(N, K) if nvfp4 else mxfp4_scale_bytes(N, K)
    w = [_address("codes", codes, device, torch.uint8, E * N * (K // 2)),
         _address("scales", scales, device, torch.uint8, E * per)]
    if nvfp4:
        if global_scales is None:
            raise ValueError("NVFP4 weights have a global scale")
        w.append(_address("global_scales", global_scales, device, torch.float32, 4 * E))
    return f16, device, xa, ya, w, N


def _matvec(x, codes, scales, global_scale, y, stream, nvfp4):
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K/2]")
    f16, device, xa, ya, w, N = _product(x, codes, scales, global_scale, y, 1, nvfp4)
    if ya[1] != xa[1]:
        raise ValueError(f"y must have {xa[1]} rows, got {ya[1]}")
    _decode_call(("matvec", nvfp4, f16), device, stream,
                 (*xa, *w, N, ya[0], ya[3], y.dtype is torch.float32))


def mxfp4_matvec(x, codes, scales, y, stream=None) -> None:
    """``y`` [T, N] = ``x`` [T, K] (BF16 or FP16) times the transpose of the
    MXFP4 weights ``codes`` [N, K/2] with tiled ``scales``; ``y`` of x's type
    or float32.  Made for few tokens."""
    _matvec(x, codes, scales, None, y, stream, False)


def mxfp4_matvec_nvfp4(x, codes, scales, global_scale, y, stream=None) -> None:
    """mxfp4_matvec with NVFP4 weights (float32 device ``global_scale``)."""
    _matvec(x, codes, scales, global_scale, y, stream, True)


def _moe_matvec(x, row_index, expert_offsets, codes, scales, global_scales, y, status, stream,
                nvfp4):
    if codes.dim() != 3:
        raise ValueError("codes must be [E, N, K/2]")
    E = codes.shape[0]
    f16, device, xa, ya, w, N = _product(x, codes, scales, global_scales, y, E, nvfp4)
    rows = ya[1]
    offsets = _address("expert_offsets", expert_offsets, device, torch.int32, 4 * (E + 1))
    index = _address("row_index", row_index, device, torch.int32, 4 * rows)
    if index is None and xa[1] < rows:
        raise ValueError(f"x holds {xa[1]} rows; without row_index this call needs {rows}")
    _decode_call(("moe_matvec", nvfp4, f16), device, stream,
                 (*xa, index, rows, offsets, E, *w, N, ya[0], ya[3], y.dtype is torch.float32,
                  _address("status", status, device, torch.int32, 4)))


def mxfp4_moe_matvec(x, row_index, expert_offsets, codes, scales, y, status=None,
                     stream=None) -> None:
    """The experts' products: row r of segment e (``expert_offsets`` int32
    [E+1]) of the routed batch is ``x[row_index[r]]`` (or ``x[r]`` without
    ``row_index``) times the transpose of expert e's MXFP4 weights ``codes``
    [E, N, K/2].  Rows of ``y`` from expert_offsets[E] on are not written."""
    _moe_matvec(x, row_index, expert_offsets, codes, scales, None, y, status, stream, False)


def mxfp4_moe_matvec_nvfp4(x, row_index, expert_offsets, codes, scales, global_scales, y,
                           status=None, stream=None) -> None:
    """mxfp4_moe_matvec with NVFP4 weights (float32 ``global_scales`` [E])."""
    _moe_matvec(x, row_index, expert_offsets, codes, scales, global_scales, y, status, stream,
                True)


# ------------------------------------------------------ the paged 4-bit cache
class KVCache(NamedTuple):
    """A paged cache of keys and values: uint8 codes [pages, heads, page_size,
    head_dim/2] and scales [pages, heads, page_size, head_dim/32 (MXFP4) or
    head_dim/16 (NVFP4)].  An NVFP4 cache has the float32 device scalars
    ``k_global`` and ``v_global``; an MXFP4 cache has None there."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_global: Optional[torch.Tensor] = None
    v_global: Optional[torch.Tensor] = None


def _cache(c, device):
    """(shape, addresses of codes and scales, of the global scales) of a cache
    whose tensors fit together."""
    k_codes, k_scales, v_codes, v_scales, k_global, v_global = c
    nvfp4 = k_global is not None
    if nvfp4 != (v_global is not None):
        raise ValueError("an NVFP4 cache has both k_global and v_global, an MXFP4 cache neither")
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [pages, heads, page_size, head_dim/2]")
    shape = pages, heads, page_size, half = k_codes.shape
    per = 8 if nvfp4 else 16
    if v_codes.shape != shape:
        raise ValueError(f"v_codes must be {tuple(shape)}, got {tuple(v_codes.shape)}")
    want = (pages, heads, page_size, half // per)
    if k_scales.shape != want or v_scales.shape != want:
        raise ValueError(f"k_scales and v_scales must be {want}")
    u8 = torch.uint8
    for t in (k_codes, k_scales, v_codes, v_scales):
        if t.get_device() != device or t.dtype is not u8 or not t.is_contiguous():
            for name in KVCache._fields[:4]:  # says which and why
                _address(name, getattr(c, name), device, u8, 0)
    tensors = (k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr())
    scalars = (_address("k_global", k_global, device, torch.float32, 4),
               _address("v_global", v_global, device, torch.float32, 4)) if nvfp4 else ()
    return pages, heads, page_size, 2 * half, tensors, scalars


def _strided(name, t, device, dtype, shape):
    """(address, outer strides) of a 3-D tensor with unit element stride; a
    dimension of one, which may report any stride, has 0."""
    if _device_index(name, t) != device:
        raise ValueError(f"all tensors must be on the same CUDA device, {name} is on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    a, b, c = t.stride()
    if c != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit element stride")
    return t.data_ptr(), (a if shape[0] > 1 else 0, b if shape[1] > 1 else 0)


def mxfp4_cache_write(k, v, slots, cache, status=None, stream=None) -> None:
    """Quantize ``k`` and ``v`` [T, heads, head_dim] (BF16 or FP16, any token
    and head stride that is a multiple of 8) into the slots ``slots`` (int32
    [T], -1: not written) of ``cache``."""
    device = _device_index("k", k)
    f16 = _half_type("k", k)
    pages, heads, page_size, D, tensors, scalars = _cache(cache, device)
    T = slots.numel()
    shape = (T, heads, D)
    ka, ks = _strided("k", k, device, k.dtype, shape)
    va, vs = _strided("v", v, device, k.dtype, shape)
    _decode_call(("cache_write", len(scalars) > 0, f16), device, stream,
                 (ka, va, T, heads, D, *ks, *vs, _address("slots", slots, device, torch.int32, 0),
                  pages, page_size, *scalars, *tensors,
                  _address("status", status, device, torch.int32, 4)))


def mxfp4_cache_read(cache, slots, k_out, v_out, status=None, stream=None) -> None:
    """Dequantize the slots ``slots`` (int32 [T], -1: zeros) of ``cache`` into
    contiguous ``k_out`` and ``v_out`` [T, heads, head_dim] (BF16 or FP16)."""
    device = _device_index("k_out", k_out)
    f16 = _half_type("k_out", k_out)
    pages, heads, page_size, D, tensors, scalars = _cache(cache, device)
    T = slots.numel()
    nbytes = 2 * T * heads * D
    _decode_call(("cache_read", len(scalars) > 0, f16), device, stream,
                 (*tensors, *scalars, pages, page_size, heads, D,
                  _address("slots", slots, device, torch.int32, 0), T,
                  _address("k_out", k_out, device, k_out.dtype, nbytes),
                  _address("v_out", v_out, device, k_out.dtype, nbytes),
                  _address("status", status, device, torch.int32, 4)))


@functools.lru_cache(maxsize=1024)
def _attention_workspace_bytes(device, *sizes) -> int:
    """The query on ``device`` (an index; None: the one that no call has changed)."""
    if device is None or device == _get_device():
        return int(_lib.mxfp4_cache_attention_workspace_bytes(*map(int, sizes)))
    with torch.cuda.device(device):
        return int(_lib.mxfp4_cache_attention_workspace_bytes(*map(int, sizes)))


def mxfp4_cache_attention_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                          head_dim: int, page_size: int, max_pages: int) -> int:
    """Bytes of workspace on the current device."""
    return _attention_workspace_bytes(_get_device() if torch.cuda.is_initialized() else None, num_seqs,
                                      num_q_heads, num_kv_heads, head_dim, page_size, max_pages)


def mxfp4_cache_attention(q, cache, page_table, seq_lens, softmax_scale: float, out, window=0,
                          workspace=None, lse=None, status=None, stream=None) -> None:
    """Attention of one query token per sequence, ``q`` [B, q_heads, head_dim]
    (BF16 or FP16), over ``cache``: sequence b's position j is in page
    ``page_table[b, j // page_size]`` (int32 [B, max_pages]), its length
    ``seq_lens[b]`` (int32).  ``window`` > 0 keeps the last ``window``
    positions.  ``workspace``: >= mxfp4_cache_attention_workspace_bytes bytes;
    ``lse``: float32 [B, q_heads]."""
    device = _device_index("q", q)
    f16 = _half_type("q", q)
    pages, heads, page_size, D, tensors, scalars = _cache(cache, device)
    if q.dim() != 3:
        raise ValueError(f"q must be [sequences, heads, {D}]")
    B, Hq, _ = q.shape
    qa, qs = _strided("q", q, device, q.dtype, (B, Hq, D))
    table = _matrix("page_table", page_table, device, (torch.int32,))
    if table[1] != B:
        raise ValueError(f"page_table must have {B} rows, got {table[1]}")
    ws = _address("workspace", workspace, device, None, 0)
    _decode_call(("cache_attention", len(scalars) > 0, f16), device, stream,
                 (qa, B, Hq, D, *qs, *tensors, *scalars, pages, page_size, heads, table[0],
                  table[3], table[2], _address("seq_lens", seq_lens, device, torch.int32, 4 * B),
                  softmax_scale, window, ws,
                  0 if ws is None else workspace.numel() * workspace.element_size(),
                  _address("out", out, device, q.dtype, 2 * B * Hq * D),
                  _address("lse", lse, device, torch.float32, 4 * B * Hq),
                  _address("status", status, device, torch.int32, 4)))


# ------------------------------------------ a layer's products, many tokens
_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}
_GATES = {None: 0, "first": 1, "second": 2}
_GROUP_SCORES = {"max": 0, "sum2": 1}


def _choice(name, value, choices):
    try:
        return choices[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {tuple(choices)}, got {value!r}") from None


def mxfp4_moe_topk(logits, top_k: int, ids, weights, score="softmax", bias=None, groups=1,
                   top_groups=1, group_score="max", renormalize=True, scale=1.0,
                   stream=None) -> None:
    """The router's choice from ``logits`` [T, E] (BF16, FP16 or float32; row
    stride may exceed E): ``ids`` int32 [T, top_k] and ``weights`` float32
    [T, top_k].  ``score``: "softmax" or "sigmoid"; ``bias`` (float32 [E]) is
    added for the choice only; ``groups`` of consecutive experts, of which the
    ``top_groups`` best by their best expert (``group_score`` "max") or the sum
    of their two best ("sum2") stay.  Weights are the chosen scores, divided by
    their sum with ``renormalize``, times ``scale``.  Equal ones go to the lowest
    index; logits that are not finite are out; -1 where no expert is left."""
    device = _device_index("logits", logits)
    la, T, E, ld = _matrix("logits", logits, device, (torch.bfloat16, torch.float16, torch.float32))
    n = 4 * T * top_k
    _launch(_lib.layer["moe_topk", logits.dtype], device, stream,
            (la, T, E, ld, _address("bias", bias, device, torch.float32, 4 * E),
             _choice("score", score, _SCORES), groups, top_groups,
             _choice("group_score", group_score, _GROUP_SCORES), top_k, bool(renormalize), scale,
             _address("ids", ids, device, torch.int32, n),
             _address("weights", weights, device, torch.float32, n)))


def _layer_product(x_codes, x_scales, x_globals, codes, scales, globals_, bias, activation, gate,
                   y, rows_of_scales, E, nvfp4):
    """The checked arguments that the dense and the experts' products share:
    (FP16, device, x's, K, the weights', the epilogue's, y's address, rows,
    columns and stride)."""
    device = _device_index("x_codes", x_codes)
    f16 = _half_type("y", y)
    if x_codes.dim() != 2:
        raise ValueError("x_codes must be [rows, K/2]")
    rows, half = x_codes.shape
    K, N = 2 * half, codes.shape[-2]
    if codes.shape[-1] != half:
        raise ValueError(f"codes hold {codes.shape[-1] * 2} elements per row, x_codes {K}")
    ya = _matrix("y", y, device, (y.dtype,))
    gate = _choice("gate", gate, _GATES)
    cols = N // 2 if gate else N
    if ya[1] != rows or ya[2] != cols:
        raise ValueError(f"y must be [{rows}, {cols}], got [{ya[1]}, {ya[2]}]")
    per = mxfp4_nvfp4_scale_bytes(N, K) if nvfp4 else mxfp4_scale_bytes(N, K)
    u8 = torch.uint8
    x = [_address("x_codes", x_codes, device, u8, 0),
         _address("x_scales", x_scales, device, u8, rows_of_scales(rows, K))]
    w = [_address("codes", codes, device, u8, E * N * half),
         _address("scales", scales, device, u8, E * per)]
    if nvfp4:
        for name, g, to in (("x_global_scale", x_globals, x), ("global_scale", globals_, w)):
            if g is None:
                raise ValueError(f"NVFP4 operands have a {name}")
            to.append(_address(name, g, device, torch.float32, 4 * E))
    epilogue = (_address("bias", bias, device, y.dtype, 2 * E * N),
                _choice("activation", activation, _ACTIVATIONS), gate)
    return f16, device, x, K, w, N, epilogue, ya


def _gemm(x_codes, x_scales, x_global, codes, scales, global_scale, y, bias, activation, gate,
          residual, stream, nvfp4):
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K/2]")
    f16, device, x, K, w, N, epilogue, ya = _layer_product(
        x_codes, x_scales, x_global, codes, scales, global_scale, bias, activation, gate, y,
        mxfp4_nvfp4_scale_bytes if nvfp4 else mxfp4_scale_bytes, 1, nvfp4)
    ra = (None, 0, 0, 0)
    if residual is not None:
        ra = _matrix("residual", residual, device, (y.dtype,))
        if ra[1] != ya[1] or ra[2] != ya[2]:
            raise ValueError(f"residual must be [{ya[1]}, {ya[2]}], got [{ra[1]}, {ra[2]}]")
    _launch(_lib.layer["gemm", nvfp4, f16], device, stream,
            (*x, ya[1], K, *w, N, *epilogue, ra[0], ra[3], ya[0], ya[3]))


def mxfp4_gemm(x_codes, x_scales, codes, scales, y, bias=None, activation=None, gate=None,
               residual=None, stream=None) -> None:
    """``y`` [T, N] = act(X W^T + ``bias``) + ``residual`` with MXFP4 X
    (``x_codes`` [T, K/2], tiled ``x_scales``) and W (``codes`` [N, K/2],
    ``scales``), as the quantize calls write them.  ``activation``: None,
    "silu", "gelu" or "gelu_tanh"; ``gate`` "first" or "second": W's rows are
    two halves, that one is activated and multiplies the other, y is
    [T, N/2].  ``y``, ``bias`` and ``residual`` are all BF16 or all FP16;
    ``residual`` may be ``y``."""
    _gemm(x_codes, x_scales, None, codes, scales, None, y, bias, activation, gate, residual,
          stream, False)


def mxfp4_gemm_nvfp4(x_codes, x_scales, x_global_scale, codes, scales, global_scale, y, bias=None,
                     activation=None, gate=None, residual=None, stream=None) -> None:
    """mxfp4_gemm with NVFP4 operands and their float32 device global scales."""
    _gemm(x_codes, x_scales, x_global_scale, codes, scales, global_scale, y, bias, activation,
          gate, residual, stream, True)


def _moe_gemm(x_codes, x_scales, x_globals, expert_offsets, codes, scales, globals_, y, bias,
              activation, gate, status, stream, nvfp4):
    if codes.dim() != 3:
        raise ValueError("codes must be [E, N, K/2]")
    E = codes.shape[0]
    bound = mxfp4_nvfp4_grouped_scale_bytes_bound if nvfp4 else mxfp4_grouped_scale_bytes_bound
    f16, device, x, K, w, N, epilogue, ya = _layer_product(
        x_codes, x_scales, x_globals, codes, scales, globals_, bias, activation, gate, y,
        lambda rows, k: bound(rows, E, k), E, nvfp4)
    offsets = _address("expert_offsets", expert_offsets, device, torch.int32, 4 * (E + 1))
    _launch(_lib.layer["moe_gemm", nvfp4, f16], device, stream,
            (*x, ya[1], K, offsets, E, *w, N, *epilogue, ya[0], ya[3],
             _address("status", status, device, torch.int32, 4)))


def mxfp4_moe_gemm(x_codes, x_scales, expert_offsets, codes, scales, y, bias=None, activation=None,
                   gate=None, status=None, stream=None) -> None:
    """The experts' products of a routed batch: row r of segment e
    (``expert_offsets`` int32 [E+1]) of the MXFP4 ``x_codes`` [rows, K/2] and
    ``x_scales`` (as the grouped quantize calls write them) with expert e's
    weights ``codes`` [E, N, K/2] and ``bias`` [E, N], as mxfp4_gemm.  Rows of
    ``y`` from expert_offsets[E] on are not written."""
    _moe_gemm(x_codes, x_scales, None, expert_offsets, codes, scales, None, y, bias, activation,
              gate, status, stream, False)


def mxfp4_moe_gemm_nvfp4(x_codes, x_scales, x_global_scales, expert_offsets, codes, scales,
                         global_scales, y, bias=None, activation=None, gate=None, status=None,
                         stream=None) -> None:
    """mxfp4_moe_gemm with NVFP4 operands (float32 global scales [E] each)."""
    _moe_gemm(x_codes, x_scales, x_global_scales, expert_offsets, codes, scales, global_scales, y,
              bias, activation, gate, status, stream, True)


def mxfp4_moe_combine(rows, dest_rows, weights, y, residual=None, status=None,
                      stream=None) -> None:
    """``y`` [T, N] (BF16 or FP16) = ``residual`` + the sum over j of
    ``weights[t, j] * rows[dest_rows[t, j]]``: ``rows`` [R, N] of y's type or
    float32, ``dest_rows`` int32 [T, top_k] (-1: nothing), ``weights`` float32
    [T, top_k].  ``residual`` may be ``y``."""
    device = _device_index("rows", rows)
    f16 = _half_type("y", y)
    a = _matrix("rows", rows, device, (y.dtype, torch.float32))
    ya = _matrix("y", y, device, (y.dtype,))
    if dest_rows.dim() != 2:
        raise ValueError("dest_rows must be [T, top_k]")
    T, top_k = dest_rows.shape
    if ya[1] != T or ya[2] != a[2]:
        raise ValueError(f"y must be [{T}, {a[2]}], got [{ya[1]}, {ya[2]}]")
    ra = (None, 0, 0, 0)
    if residual is not None:
        ra = _matrix("residual", residual, device, (y.dtype,))
        if ra[1] != T or ra[2] != ya[2]:
            raise ValueError(f"residual must be [{T}, {ya[2]}], got [{ra[1]}, {ra[2]}]")
    _launch(_lib.layer["moe_combine", f16], device, stream,
            (a[0], rows.dtype is torch.float32, a[1], a[2], a[3],
             _address("dest_rows", dest_rows, device, torch.int32, 0),
             _address("weights", weights, device, torch.float32, 4 * T * top_k), T, top_k, ra[0],
             ra[3], ya[0], ya[3], _address("status", status, device, torch.int32, 4)))


# --------------------------------------------------- allocating wrappers
def _empty(shape, dtype, device, stream, make=torch.empty):
    """An uninitialised (``make`` torch.zeros: zeroed there) tensor for a call on
    ``stream`` (None: the current one).  Memory is a stream's: a block that was
    freed on the current stream may still be in use there, and one freed here
    goes to the current stream's next tensor, so what the call on another stream
    writes is that stream's memory.  It may be used and freed on the current
    stream as well."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def quantize(x, stream=None):
    """BF16 or FP16 ``x`` [M, K] -> (codes uint8 [M, K/2], scales uint8 [scale_bytes])."""
    M, K = x.shape
    codes = _empty((M, K // 2), torch.uint8, x.device, stream)
    scales = _empty(mxfp4_scale_bytes(M, K), torch.uint8, x.device, stream)
    if x.dtype == torch.float16:
        mxfp4_quantize_f16(x, codes, scales, stream)
    else:
        mxfp4_quantize(x, codes, scales, stream)
    return codes, scales


def quantize_grouped(x, expert_offsets, stream=None):
    """Returns (codes, scales, scale_row_offsets int32 [E+1], status int32 [1])."""
    total, K = x.shape
    E = expert_offsets.numel() - 1
    dev = x.device
    codes = _empty((total, K // 2), torch.uint8, dev, stream)
    scales = _empty(max(mxfp4_grouped_scale_bytes_bound(total, E, K), 16),
                    torch.uint8, dev, stream)
    sro = _empty(E + 1, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    _grouped(x, expert_offsets, codes, scales, sro, status, stream, x.dtype == torch.float16)
    return codes, scales, sro, status


def quantize_grouped_gather(x, row_index, expert_offsets, stream=None, via_scatter=True):
    """Returns (codes, scales, scale_row_offsets, status) of x[row_index]
    (BF16 or FP16 x).  By default through the scatter path, with a workspace
    allocated here; via_scatter=False calls the entry point without a
    workspace, which borrows the tail of its codes output as one when that
    fits and otherwise runs the per-row gather kernel (same results)."""
    K = x.shape[1]
    total = row_index.numel()
    E = expert_offsets.numel() - 1
    dev = x.device
    f16 = x.dtype == torch.float16
    codes = _empty((total, K // 2), torch.uint8, dev, stream)
    scales = _empty(max(mxfp4_grouped_scale_bytes_bound(total, E, K), 16),
                    torch.uint8, dev, stream)
    sro = _empty(E + 1, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    if via_scatter:
        ws = _empty(max(mxfp4_gather_workspace_bytes(x.shape[0], total, E, K), 16),
                    torch.uint8, dev, stream)
        _gather_ws(x, row_index, expert_offsets, ws, codes, scales, sro, status, stream, f16)
    else:
        _gather(x, row_index, expert_offsets, codes, scales, sro, status, stream, f16)
    return codes, scales, sro, status


def quantize_grouped_scatter(x, dest_rows, expert_offsets, total_rows=None, stream=None,
                             staged=True):
    """Returns (codes, scales, scale_row_offsets, status) of the expert-sorted
    batch that ``dest_rows`` dispatches ``x`` into.  ``total_rows`` defaults
    to ``dest_rows.numel()`` (every route dispatched); rows that no route
    targets come back zero.  By default each token's scale words are staged
    in a workspace allocated here (same results); staged=False stores every
    route's scale words directly."""
    K = x.shape[1]
    total = dest_rows.numel() if total_rows is None else int(total_rows)
    E = expert_offsets.numel() - 1
    dev = x.device
    codes = _empty((total, K // 2), torch.uint8, dev, stream, torch.zeros)
    scales = _empty(max(mxfp4_grouped_scale_bytes_bound(total, E, K), 16),
                    torch.uint8, dev, stream, torch.zeros)
    sro = _empty(E + 1, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    ws = None
    if staged:
        ws = _empty(max(mxfp4_scatter_workspace_bytes(x.shape[0], total, E, K), 16),
                    torch.uint8, dev, stream)
    _scatter(x, dest_rows, expert_offsets, total, codes, scales, sro, status, stream,
             x.dtype == torch.float16, ws)
    return codes, scales, sro, status


def moe_route(topk_ids, num_experts: int, stream=None):
    """Returns (expert_offsets, dest_rows, row_index, status) of the router's
    expert ids ``topk_ids`` [num_tokens, top_k]: the inputs of the grouped,
    scatter and gather calls (row_index holds expert_offsets[-1] valid rows;
    the rest of it is not written)."""
    dev = topk_ids.device
    T, top_k = topk_ids.shape
    off = _empty(num_experts + 1, torch.int32, dev, stream)
    dest = _empty((T, top_k), torch.int32, dev, stream)
    rows = _empty(max(T * top_k, 1), torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    ws = _empty(max(mxfp4_route_workspace_bytes(T, top_k, num_experts), 16),
                torch.uint8, dev, stream)
    mxfp4_moe_route(topk_ids, num_experts, ws, off, dest, rows, status, stream)
    return off, dest, rows, status


def dequantize(codes, scales, M: int, K: int, stream=None):
    y = _empty((M, K), torch.bfloat16, codes.device, stream)
    mxfp4_dequantize(codes, scales, M, K, y, stream)
    return y


def swap_w13(codes, scales, w13_bias=None, w2_bias=None, scales_tiled=True, stream=None):
    """codes uint8 [E, 2N, K/2]; scales tiled (E x scale_bytes(2N, K)) or flat
    [E, 2N, K/32].  Returns (codes, scales, w13_bias_bf16, w2_bias_bf16)."""
    E, two_n, half_k = codes.shape
    K = half_k * 2
    codes_out = _empty(codes.shape, codes.dtype, codes.device, stream)
    scales_out = _empty(scales.shape, scales.dtype, scales.device, stream)
    b13 = _empty(w13_bias.shape, torch.bfloat16, codes.device, stream) \
        if w13_bias is not None else None
    b2 = _empty(w2_bias.shape, torch.bfloat16, codes.device, stream) \
        if w2_bias is not None else None
    mxfp4_swap_w13(codes, scales, w13_bias, E, two_n, K, 1 if scales_tiled else 0, codes_out,
                   scales_out, b13, w2_bias, b2, stream)
    return codes_out, scales_out, b13, b2


def quantize_nvfp4(x, global_scale, stream=None):
    """Returns (codes uint8 [M, K/2], E4M3 scales uint8 [nvfp4_scale_bytes])
    of BF16 or FP16 ``x``."""
    M, K = x.shape
    codes = _empty((M, K // 2), torch.uint8, x.device, stream)
    scales = _empty(mxfp4_nvfp4_scale_bytes(M, K), torch.uint8, x.device, stream)
    _nvfp4(x, global_scale, codes, scales, stream, x.dtype == torch.float16)
    return codes, scales


def quantize_nvfp4_grouped(x, expert_offsets, global_scales, stream=None):
    """Returns (codes, scales, scale_row_offsets, status) of the NVFP4 experts
    quant of the expert-sorted ``x`` (BF16 or FP16)."""
    total, K = x.shape
    E = expert_offsets.numel() - 1
    dev = x.device
    codes = _empty((total, K // 2), torch.uint8, dev, stream)
    scales = _empty(max(mxfp4_nvfp4_grouped_scale_bytes_bound(total, E, K), 16),
                    torch.uint8, dev, stream)
    sro = _empty(E + 1, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    _nvfp4_grouped(x, expert_offsets, global_scales, codes, scales, sro, status, stream,
                   x.dtype == torch.float16)
    return codes, scales, sro, status


def quantize_nvfp4_grouped_scatter(x, dest_rows, expert_offsets, global_scales, total_rows=None,
                                   stream=None, staged=True):
    """Returns (codes, scales, scale_row_offsets, status) of the NVFP4 experts
    quant of the batch ``dest_rows`` dispatches ``x`` (BF16 or FP16) into;
    rows no route targets come back zero.  By default the scale bytes are
    staged in a workspace allocated here (same results); staged=False stores
    each route's scale words straight into the tiled layout."""
    K = x.shape[1]
    total = dest_rows.numel() if total_rows is None else int(total_rows)
    E = expert_offsets.numel() - 1
    dev = x.device
    codes = _empty((total, K // 2), torch.uint8, dev, stream, torch.zeros)
    scales = _empty(max(mxfp4_nvfp4_grouped_scale_bytes_bound(total, E, K), 16),
                    torch.uint8, dev, stream, torch.zeros)
    sro = _empty(E + 1, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream)
    ws = None
    if staged:
        ws = _empty(max(mxfp4_nvfp4_scatter_workspace_bytes(total, E, K), 16),
                    torch.uint8, dev, stream)
    _nvfp4_scatter(x, dest_rows, expert_offsets, total, global_scales, codes, scales, sro, status,
                   stream, x.dtype == torch.float16, ws)
    return codes, scales, sro, status


def dequantize_nvfp4(codes, scales, global_scale, M: int, K: int, stream=None):
    y = _empty((M, K), torch.bfloat16, codes.device, stream)
    mxfp4_dequantize_nvfp4(codes, scales, global_scale, M, K, y, stream)
    return y


def _product_out(x, rows, N, out, out_dtype, stream):
    return out if out is not None else _empty((rows, N), out_dtype or x.dtype, x.device, stream)


def matvec(x, codes, scales, out=None, out_dtype=None, stream=None):
    """``x`` [T, K] (BF16 or FP16) times the transpose of the MXFP4 weights
    ``codes`` [N, K/2], ``scales`` (tiled): [T, N] of x's type, of
    ``out_dtype`` (torch.float32) or into ``out``."""
    out = _product_out(x, x.shape[0], codes.shape[0], out, out_dtype, stream)
    _matvec(x, codes, scales, None, out, stream, False)
    return out


def matvec_nvfp4(x, codes, scales, global_scale, out=None, out_dtype=None, stream=None):
    """matvec with NVFP4 weights and their float32 ``global_scale``."""
    out = _product_out(x, x.shape[0], codes.shape[0], out, out_dtype, stream)
    _matvec(x, codes, scales, global_scale, out, stream, True)
    return out


def _moe_outputs(x, row_index, codes, out, out_dtype, status, stream):
    rows = x.shape[0] if row_index is None else row_index.numel()
    if status is None:
        status = _empty(1, torch.int32, x.device, stream)
    return _product_out(x, rows, codes.shape[1], out, out_dtype, stream), status


def moe_matvec(x, row_index, expert_offsets, codes, scales, out=None, out_dtype=None, status=None,
               stream=None):
    """Returns (y, status): y [rows, N], row r of segment e = x[row_index[r]]
    (x[r] if row_index is None) times the transpose of expert e's MXFP4
    weights ``codes`` [E, N, K/2].  Rows from expert_offsets[E] on are not
    written."""
    out, status = _moe_outputs(x, row_index, codes, out, out_dtype, status, stream)
    _moe_matvec(x, row_index, expert_offsets, codes, scales, None, out, status, stream, False)
    return out, status


def moe_matvec_nvfp4(x, row_index, expert_offsets, codes, scales, global_scales, out=None,
                     out_dtype=None, status=None, stream=None):
    """moe_matvec with NVFP4 weights and float32 ``global_scales`` [E]."""
    out, status = _moe_outputs(x, row_index, codes, out, out_dtype, status, stream)
    _moe_matvec(x, row_index, expert_offsets, codes, scales, global_scales, out, status, stream,
                True)
    return out, status


def cache_alloc(num_pages: int, page_size: int, num_heads: int, head_dim: int, k_global=None,
                v_global=None, device="cuda"):
    """A zeroed KVCache; NVFP4 when the float32 global scales are given."""
    per = 32 if k_global is None else 16
    shape = (num_pages, num_heads, page_size)
    parts = [torch.zeros(*shape, n, dtype=torch.uint8, device=device)
             for n in (head_dim // 2, head_dim // per) * 2]
    return KVCache(*parts, k_global, v_global)


def cache_write(k, v, slots, cache, status=None, stream=None):
    """mxfp4_cache_write with a status word allocated here; returns it."""
    if status is None:
        status = _empty(1, torch.int32, k.device, stream)
    mxfp4_cache_write(k, v, slots, cache, status, stream)
    return status


def cache_read(cache, slots, k_out=None, v_out=None, dtype=torch.bfloat16, status=None,
               stream=None):
    """Returns (k, v, status): the slots' keys and values [T, heads, head_dim]."""
    shape = (slots.numel(), cache.k_codes.shape[1], cache.k_codes.shape[3] * 2)
    k_out, v_out = (t if t is not None else _empty(shape, dtype, slots.device, stream)
                    for t in (k_out, v_out))
    if status is None:
        status = _empty(1, torch.int32, slots.device, stream)
    mxfp4_cache_read(cache, slots, k_out, v_out, status, stream)
    return k_out, v_out, status


def cache_attention(q, cache, page_table, seq_lens, softmax_scale: float, window=0, out=None,
                    lse=None, status=None, stream=None):
    """Returns (out [B, q_heads, head_dim], lse float32 [B, q_heads], status),
    with the workspace allocated here."""
    B, Hq, D = q.shape
    if out is None:
        out = _empty((B, Hq, D), q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((B, Hq), torch.float32, q.device, stream)
    if status is None:
        status = _empty(1, torch.int32, q.device, stream)
    nbytes = _attention_workspace_bytes(q.get_device(), B, Hq, cache.k_codes.shape[1], D,
                                        cache.k_codes.shape[2], page_table.shape[1])
    ws = _empty(nbytes, torch.uint8, q.device, stream) if nbytes else None
    mxfp4_cache_attention(q, cache, page_table, seq_lens, softmax_scale, out, window, ws, lse,
                          status, stream)
    return out, lse, status


def moe_topk(logits, top_k: int, score="softmax", bias=None, groups=1, top_groups=1,
             group_score="max", renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """Returns (ids int32 [T, top_k], weights float32 [T, top_k]) of the router's
    ``logits`` [T, E]; see mxfp4_moe_topk."""
    shape = (logits.shape[0], top_k)
    if ids is None:
        ids = _empty(shape, torch.int32, logits.device, stream)
    if weights is None:
        weights = _empty(shape, torch.float32, logits.device, stream)
    mxfp4_moe_topk(logits, top_k, ids, weights, score, bias, groups, top_groups, group_score,
                   renormalize, scale, stream)
    return ids, weights


def _layer_out(x_codes, codes, gate, out, out_dtype, stream):
    if out is not None:
        return out
    N = codes.shape[-2]
    return _empty((x_codes.shape[0], N if gate is None else N // 2), out_dtype, x_codes.device,
                  stream)


def gemm(x_codes, x_scales, codes, scales, bias=None, activation=None, gate=None, residual=None,
         out=None, out_dtype=torch.bfloat16, stream=None):
    """act(X W^T + bias) + residual of MXFP4 X [T, K] and W [N, K]: [T, N] (with
    a gate [T, N/2]) of ``out_dtype`` or into ``out``; see mxfp4_gemm."""
    out = _layer_out(x_codes, codes, gate, out, out_dtype, stream)
    _gemm(x_codes, x_scales, None, codes, scales, None, out, bias, activation, gate, residual,
          stream, False)
    return out


def gemm_nvfp4(x_codes, x_scales, x_global_scale, codes, scales, global_scale, bias=None,
               activation=None, gate=None, residual=None, out=None, out_dtype=torch.bfloat16,
               stream=None):
    """gemm with NVFP4 operands and their float32 global scales."""
    out = _layer_out(x_codes, codes, gate, out, out_dtype, stream)
    _gemm(x_codes, x_scales, x_global_scale, codes, scales, global_scale, out, bias, activation,
          gate, residual, stream, True)
    return out


def moe_gemm(x_codes, x_scales, expert_offsets, codes, scales, bias=None, activation=None,
             gate=None, out=None, out_dtype=torch.bfloat16, status=None, stream=None):
    """Returns (y, status) of the experts' products over a routed batch that the
    grouped quantize calls wrote; see mxfp4_moe_gemm."""
    out = _layer_out(x_codes, codes, gate, out, out_dtype, stream)
    if status is None:
        status = _empty(1, torch.int32, x_codes.device, stream)
    _moe_gemm(x_codes, x_scales, None, expert_offsets, codes, scales, None, out, bias, activation,
              gate, status, stream, False)
    return out, status


def moe_gemm_nvfp4(x_codes, x_scales, x_global_scales, expert_offsets, codes, scales,
                   global_scales, bias=None, activation=None, gate=None, out=None,
                   out_dtype=torch.bfloat16, status=None, stream=None):
    """moe_gemm with NVFP4 operands and float32 global scales [E] of each."""
    out = _layer_out(x_codes, codes, gate, out, out_dtype, stream)
    if status is None:
        status = _empty(1, torch.int32, x_codes.device, stream)
    _moe_gemm(x_codes, x_scales, x_global_scales, expert_offsets, codes, scales, global_scales,
              out, bias, activation, gate, status, stream, True)
    return out, status


def moe_combine(rows, dest_rows, weights, residual=None, out=None, out_dtype=None, status=None,
                stream=None):
    """Returns (y, status): every token's weighted sum of its experts' ``rows``,
    added to ``residual``; y of ``out_dtype`` (of residual's or rows' type, where
    that is not float32, else BF16) or into ``out``; see mxfp4_moe_combine."""
    if out is None:
        if out_dtype is None:
            out_dtype = rows.dtype if residual is None else residual.dtype
            out_dtype = torch.bfloat16 if out_dtype is torch.float32 else out_dtype
        out = _empty((dest_rows.shape[0], rows.shape[1]), out_dtype, rows.device, stream)
    if status is None:
        status = _empty(1, torch.int32, rows.device, stream)
    mxfp4_moe_combine(rows, dest_rows, weights, out, residual, status, stream)
    return out, status

// cache.cu — keys and values quantized into a paged 4-bit cache, and read
// back from it, for sm_103a.
//
// The cache holds, for keys and for values, codes [pages, heads, page_size,
// head_dim/2] and scales [pages, heads, page_size, head_dim/32 (MXFP4) or /16
// (NVFP4)].  Each (token, head) row is quantized on its own, by the rules and
// with the device code of the dense quantizers; reading back rounds as the
// dense dequantizers do.
//
// Both kernels are a pass over the data: 2 bytes of a 16-bit value against
// 17/32 (9/16) bytes of its code and share of a scale, so HBM traffic bounds
// long calls and the launch the short ones.  A thread keeps one place of a
// token's rows (keys or values, head, 16 consecutive elements: 32 bytes in, 8
// out, or the reverse) and walks over tokens with kAtOnce of them in flight, so
// that what depends on the place alone is worked out once (a place and a token to
// each thread, found by divisions: 16 tokens 10.2 us, here 6.1, events around one
// call).
// Measured, BF16 to or from MXFP4, 8 heads of 128, slots in any order: 32768
// tokens (170 MB) written in 30.1 us (5.6 TB/s) and read in 32.3 us (5.3 TB/s), 16
// tokens in 1.9 and 1.8 us of device time.  The long calls issue on 65 % of the
// cycles; reading in random order takes 32-byte sectors for 4 bytes of scales (56 MB
// from HBM where the cache's are 36).
#include <algorithm>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache_device.cuh"
#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "nvfp4_device.cuh"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // tokens in flight per thread

struct CacheParams {
  const uint8_t* __restrict__ x[2];  // write: keys, values
  uint8_t* __restrict__ out[2];      // read: keys, values
  uint8_t* __restrict__ codes[2];
  uint8_t* __restrict__ scales[2];
  const float* __restrict__ global_scales[2];
  const int32_t* __restrict__ slots;
  int32_t* __restrict__ status;
  int64_t token_stride[2];  // elements
  int64_t head_stride[2];
  int32_t num_tokens;
  int32_t num_slots;
  int32_t page_size;
  int32_t num_heads;
  int32_t head_dim;
  int32_t page_shift;     // log2 of page_size, or -1
  int32_t lanes;          // tokens side by side in a CTA (places <= kThreads), else 1
  int32_t wide;           // 32-byte accesses of the 16-bit side are aligned
  int32_t places;         // of a token: 16-element pieces of its keys and values
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgX0 = 0, kDbgX1, kDbgCodes0, kDbgCodes1, kDbgScales0, kDbgScales1, kDbgSlots, kDbgStatus };

__device__ __forceinline__ int32_t slot_at(const CacheParams& p, int64_t t) {
  const int32_t* at = p.slots + t;
  return MXFP4_IN_BOUNDS(p, kDbgSlots, at, 4) ? __ldg(at) : -1;
}

// Status word: from all the slots, by CTA 0, which does nothing else (with many
// tokens it is as long as the others' work: 16 loads in flight, and first in the
// grid so that it does not trail).  True in CTA 0 and, idle, in those above it.
__device__ __forceinline__ bool write_status(const CacheParams& p) {
  if (p.status == nullptr || blockIdx.x != 0) return false;
  if (blockIdx.y != 0) return true;
  int bad = 0;
#pragma unroll 16
  for (int64_t t = threadIdx.x; t < p.num_tokens; t += kThreads) {
    const int32_t s = slot_at(p, t);
    if (s < -1 || s >= p.num_slots) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && MXFP4_IN_BOUNDS(p, kDbgStatus, p.status, 4)) *p.status = bad ? -7 : 0;
  return true;
}

// One place of a token: part (0 keys, 1 values), head, 16-element segment.
struct Place {
  int part, head, seg;
};
__device__ __forceinline__ Place place_of(const CacheParams& p, int place) {
  const int segs = p.head_dim / kElems;
  Place r;
  const int row = place / segs;
  r.seg = place - row * segs;
  r.part = row >= p.num_heads;
  r.head = row - (r.part ? p.num_heads : 0);
  return r;
}

// Row of the cache that (slot, head) names: (page * heads + head) * page_size + position.
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int32_t slot, int head) {
  const int32_t page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
  return (static_cast<int64_t>(page) * p.num_heads + head) * p.page_size + (slot - page * p.page_size);
}

// Every (token, place) of the call: `body(place, slots, tokens)` takes kAtOnce
// tokens of a place (slot -1: none).  All lanes of a warp make each call.
template <typename Body>
__device__ __forceinline__ void for_places(const CacheParams& p, Body body) {
  const int places = p.lanes > 1 ? p.places : kThreads;
  const int lane_token = threadIdx.x / places;
  const int word = p.status != nullptr;  // CTA 0's
  const int64_t ctas = gridDim.x - word;
  const int64_t stride = ctas * p.lanes;
  for (int u0 = blockIdx.y * kThreads; u0 < p.places; u0 += gridDim.y * kThreads) {
    const int u = u0 + threadIdx.x - lane_token * places;
    const bool live = lane_token < p.lanes && u < p.places;
    const Place place = place_of(p, live ? u : 0);
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x - word) * p.lanes; t0 < p.num_tokens; t0 += kAtOnce * stride) {
      int32_t slots[kAtOnce];
      int32_t tokens[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t t = t0 + i * stride + lane_token;
        tokens[i] = live && t < p.num_tokens ? static_cast<int32_t>(t) : -1;
        slots[i] = -1;
        if (tokens[i] >= 0) {
          const int32_t s = slot_at(p, t);
          slots[i] = s < p.num_slots ? s : -1;
        }
      }
      body(place, slots, tokens);
    }
  }
}

template <bool kNv, bool kF16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheParams p) {
  pdl_wait();
  pdl_release();
  if (write_status(p)) return;
  float g[2] = {1.0f, 1.0f};
  if constexpr (kNv) {
    g[0] = global_scale_or_one(p.global_scales[0]);
    g[1] = global_scale_or_one(p.global_scales[1]);
  }
  for_places(p, [&](const Place& w, const int32_t (&slots)[kAtOnce], const int32_t (&tokens)[kAtOnce]) {
    uint4 v[kAtOnce][2];
    const uint8_t* const x = (w.part ? p.x[1] : p.x[0]) + (w.head * (w.part ? p.head_stride[1] : p.head_stride[0]) +
                                                            w.seg * kElems) * 2;
    const int64_t token_bytes = (w.part ? p.token_stride[1] : p.token_stride[0]) * 2;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
      const uint8_t* src = x + tokens[i] * token_bytes;
      if (slots[i] >= 0 && MXFP4_IN_BOUNDS(p, kDbgX0 + w.part, src, 32)) {
        if (p.wide) load32<true>(src, v[i]); else load32<false>(src, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      uint32_t s;
      uint2 code;
      if constexpr (kNv) {
        const float gs = w.part ? g[1] : g[0];
        s = nv_scale_byte<kF16>(v[i], gs);
        code = nv_codes<kF16>(v[i], s, gs / e4m3_to_f32(s));
      } else {
        s = lane_block_scale<kF16>(v[i]);  // shared with the neighbour lane
        code = lane_codes<kF16>(v[i], s);
      }
      if (slots[i] < 0) continue;
      const int64_t row = cache_row(p, slots[i], w.head);
      uint8_t* cp = (w.part ? p.codes[1] : p.codes[0]) + row * (p.head_dim / 2) + w.seg * 8;
      if (MXFP4_IN_BOUNDS(p, kDbgCodes0 + w.part, cp, 8)) *reinterpret_cast<uint2*>(cp) = code;
      if (kNv || (w.seg & 1) == 0) {
        uint8_t* sp = (w.part ? p.scales[1] : p.scales[0]) + row * (p.head_dim / (kNv ? 16 : 32)) +
                      (kNv ? w.seg : w.seg >> 1);
        if (MXFP4_IN_BOUNDS(p, kDbgScales0 + w.part, sp, 1)) *sp = static_cast<uint8_t>(s);
      }
    }
  });
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return cvt_bf16x2(lo, hi);
  }
}

// 4 code bytes -> 8 values: MXFP4 e2m1 * sc; NVFP4 (e2m1 * sc) * inv.
template <bool kNv, bool kF16>
__device__ __forceinline__ uint4 decode8(uint32_t c, float sc, float inv) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = cvt_e2m1x2_to_f16x2(c >> (8 * i));
    float lo = half_lo_to_f32(h) * sc, hi = half_hi_to_f32(h) * sc;
    if constexpr (kNv) {
      lo *= inv;
      hi *= inv;
    }
    o[i] = pack16<kF16>(lo, hi);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kNv, bool kF16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheParams p) {
  pdl_wait();
  pdl_release();
  if (write_status(p)) return;
  float inv[2] = {1.0f, 1.0f};
  if constexpr (kNv) {
    inv[0] = 1.0f / global_scale_or_one(p.global_scales[0]);
    inv[1] = 1.0f / global_scale_or_one(p.global_scales[1]);
  }
  for_places(p, [&](const Place& w, const int32_t (&slots)[kAtOnce], const int32_t (&tokens)[kAtOnce]) {
    uint2 c[kAtOnce];
    uint32_t s[kAtOnce];
    const uint8_t* const codes = (w.part ? p.codes[1] : p.codes[0]) + w.seg * 8;
    const uint8_t* const scales = (w.part ? p.scales[1] : p.scales[0]) + (kNv ? w.seg : w.seg >> 1);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      c[i] = make_uint2(0u, 0u);
      s[i] = 0u;
      if (slots[i] < 0) continue;
      const int64_t row = cache_row(p, slots[i], w.head);
      const uint8_t* cp = codes + row * (p.head_dim / 2);
      const uint8_t* sp = scales + row * (p.head_dim / (kNv ? 16 : 32));
      if (MXFP4_IN_BOUNDS(p, kDbgCodes0 + w.part, cp, 8) && MXFP4_IN_BOUNDS(p, kDbgScales0 + w.part, sp, 1)) {
        c[i] = ld_stream_v2(cp);
        s[i] = __ldg(sp);
      }
    }
    uint8_t* const out = (w.part ? p.out[1] : p.out[0]) + (w.head * p.head_dim + w.seg * kElems) * 2;
    const int64_t token_bytes = static_cast<int64_t>(p.num_heads) * p.head_dim * 2;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (tokens[i] < 0) continue;
      uint4 o0, o1;
      if (kNv ? (s[i] & 0x7Fu) == 0x7Fu : s[i] == 255u) {
        const uint32_t q = kF16 ? 0x7E007E00u : 0x7FC07FC0u;
        o0 = o1 = make_uint4(q, q, q, q);
      } else {
        const float sc = kNv ? e4m3_to_f32(s[i]) : scale_from_e8m0(s[i]);
        const float by = w.part ? inv[1] : inv[0];
        o0 = decode8<kNv, kF16>(c[i].x, sc, by);
        o1 = decode8<kNv, kF16>(c[i].y, sc, by);
      }
      uint8_t* dst = out + tokens[i] * token_bytes;
      if (!MXFP4_IN_BOUNDS(p, kDbgX0 + w.part, dst, 32)) continue;
      if (p.wide) {
        st_stream_v8(dst, o0, o1);
      } else {
        st_stream_v4(dst, o0);
        st_stream_v4(dst + 16, o1);
      }
    }
  });
}

CacheParams cache_params(const CacheArgs& c, const int32_t* slots, int64_t num_tokens,
                         int32_t* status) {
  CacheParams p{};
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = c.codes[i];
    p.scales[i] = c.scales[i];
    p.global_scales[i] = c.global_scales[i];
  }
  p.slots = slots;
  p.status = status;
  p.num_tokens = static_cast<int32_t>(num_tokens);
  p.num_slots = static_cast<int32_t>(c.num_pages * c.page_size);
  p.page_size = c.page_size;
  p.num_heads = c.num_heads;
  p.head_dim = c.head_dim;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c.page_size == 1 << i) p.page_shift = i;
  p.places = 2 * c.num_heads * (c.head_dim / kElems);  // a row has 2^31 elements at most
  p.lanes = p.places > 0 && p.places <= kThreads ? kThreads / p.places : 1;
#ifdef MXFP4_DEBUG_BOUNDS
  const int64_t row = static_cast<int64_t>(c.num_heads) * c.head_dim;
  for (int i = 0; i < 2; ++i) {
    debug_range(p.dbg, kDbgCodes0 + i, c.codes[i], p.num_slots * (row / 2));
    debug_range(p.dbg, kDbgScales0 + i, c.scales[i], p.num_slots * (row / (c.nvfp4 ? 16 : 32)));
  }
  debug_range(p.dbg, kDbgSlots, slots, num_tokens * 4);
  debug_range(p.dbg, kDbgStatus, status, status ? 4 : 0);
#endif
  return p;
}

// CTAs for kAtOnce tokens of each thread, and for one where that would leave SMs
// without any; one more for the status word.
dim3 grid_of(const CacheParams& p) {
  const unsigned word = p.status != nullptr;
  if (p.num_tokens == 0 || p.places == 0) return dim3(1);
  const int64_t rows = (p.places + kThreads - 1) / kThreads;
  const int64_t lanes = (static_cast<int64_t>(p.num_tokens) + p.lanes - 1) / p.lanes;
  const int64_t full = (lanes + kAtOnce - 1) / kAtOnce;
  const int64_t wide = std::min(lanes, (sm_count() + rows - 1) / rows);
  return dim3(static_cast<unsigned>(std::max(full, wide)) + word,
              static_cast<unsigned>(std::min<int64_t>(rows, 65535)));
}

}  // namespace

cudaError_t launch_cache_write(const CacheArgs& c, const void* const x[2], int64_t num_tokens,
                               const int64_t token_stride[2], const int64_t head_stride[2],
                               const int32_t* slots, int32_t* status, cudaStream_t stream) {
  CacheParams p = cache_params(c, slots, num_tokens, status);
  p.wide = 1;
  for (int i = 0; i < 2; ++i) {
    p.wide &= reinterpret_cast<uintptr_t>(x[i]) % 32 == 0 && token_stride[i] % 16 == 0 && head_stride[i] % 16 == 0;
    p.x[i] = static_cast<const uint8_t*>(x[i]);
    p.token_stride[i] = token_stride[i];
    p.head_stride[i] = head_stride[i];
#ifdef MXFP4_DEBUG_BOUNDS
    debug_range(p.dbg, kDbgX0 + i, x[i],
                num_tokens > 0 && c.num_heads > 0
                    ? ((num_tokens - 1) * token_stride[i] + (c.num_heads - 1) * head_stride[i] +
                       c.head_dim) * 2
                    : 0);
#endif
  }
  const auto kernel = c.nvfp4 ? (c.f16 ? cache_write_kernel<true, true> : cache_write_kernel<true, false>)
                              : (c.f16 ? cache_write_kernel<false, true> : cache_write_kernel<false, false>);
  return launch_pdl(kernel, grid_of(p), kThreads, 0, stream, p);
}

cudaError_t launch_cache_read(const CacheArgs& c, const int32_t* slots, int64_t num_tokens,
                              void* const out[2], int32_t* status, cudaStream_t stream) {
  CacheParams p = cache_params(c, slots, num_tokens, status);
  p.wide = 1;
  for (int i = 0; i < 2; ++i) {
    p.wide &= reinterpret_cast<uintptr_t>(out[i]) % 32 == 0;
    p.out[i] = static_cast<uint8_t*>(out[i]);
#ifdef MXFP4_DEBUG_BOUNDS
    debug_range(p.dbg, kDbgX0 + i, out[i], num_tokens * c.num_heads * c.head_dim * 2);
#endif
  }
  const auto kernel = c.nvfp4 ? (c.f16 ? cache_read_kernel<true, true> : cache_read_kernel<true, false>)
                              : (c.f16 ? cache_read_kernel<false, true> : cache_read_kernel<false, false>);
  return launch_pdl(kernel, grid_of(p), kThreads, 0, stream, p);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_cache() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

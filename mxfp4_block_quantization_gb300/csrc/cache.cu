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
// long calls and the launch the short ones.  A lane takes 16 consecutive
// elements of a row (32 bytes in, 8 out, or the reverse).
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "nvfp4_device.cuh"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;

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
  int32_t tokens_per_cta;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgX0 = 0, kDbgX1, kDbgCodes0, kDbgCodes1, kDbgScales0, kDbgScales1, kDbgSlots };

// Status word: written by the first CTA alone, from all the slots.
__device__ __forceinline__ void write_status(const CacheParams& p) {
  if (blockIdx.x != 0 || p.status == nullptr) return;
  int bad = 0;
  for (int64_t t = threadIdx.x; t < p.num_tokens; t += kThreads) {
    const int32_t s = __ldg(p.slots + t);
    if (s < -1 || s >= p.num_slots) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.status = bad ? -7 : 0;
}

// One lane's 16 elements: token, part (0 keys, 1 values), head, segment.
struct Unit {
  int token, part, head, seg;
};
__device__ __forceinline__ Unit unit_of(const CacheParams& p, int first, uint32_t u, uint32_t segs) {
  Unit r;
  r.seg = u % segs;
  u /= segs;
  r.head = u % static_cast<uint32_t>(p.num_heads);
  u /= static_cast<uint32_t>(p.num_heads);
  r.part = u & 1u;
  r.token = first + static_cast<int>(u >> 1);
  return r;
}

// Row of the cache that (slot, head) names: (page * heads + head) * page_size + position.
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int32_t slot, int head) {
  const int32_t page = slot / p.page_size;
  return (static_cast<int64_t>(page) * p.num_heads + head) * p.page_size + (slot - page * p.page_size);
}

template <bool kNv, bool kF16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheParams p) {
  pdl_wait();
  pdl_release();
  write_status(p);
  const int first = blockIdx.x * p.tokens_per_cta;
  const int avail = p.num_tokens - first;
  const int tokens = avail < p.tokens_per_cta ? avail : p.tokens_per_cta;
  const uint32_t segs = p.head_dim / kElems;
  const uint32_t units = static_cast<uint32_t>(tokens) * 2u * p.num_heads * segs;
  for (uint32_t u0 = 0; u0 < units; u0 += kThreads) {
    const uint32_t u = u0 + threadIdx.x;
    const Unit w = unit_of(p, first, u < units ? u : 0u, segs);
    const int32_t slot = __ldg(p.slots + w.token);
    const bool live = u < units && slot >= 0 && slot < p.num_slots;
    uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    const uint8_t* src = p.x[w.part] + (w.token * p.token_stride[w.part] +
                                        w.head * p.head_stride[w.part] + w.seg * kElems) * 2;
    if (live && MXFP4_IN_BOUNDS(p, kDbgX0 + w.part, src, 32)) load32<false>(src, v);
    uint32_t s;
    uint2 code;
    if constexpr (kNv) {
      const float g = __ldg(p.global_scales[w.part]);
      s = nv_scale_byte<kF16>(v, g);
      code = nv_codes<kF16>(v, s, g / e4m3_to_f32(s));
    } else {
      s = lane_block_scale<kF16>(v);
      code = lane_codes<kF16>(v, s);
    }
    if (!live) continue;
    const int64_t row = cache_row(p, slot, w.head);
    uint8_t* cp = p.codes[w.part] + row * (p.head_dim / 2) + w.seg * 8;
    if (MXFP4_IN_BOUNDS(p, kDbgCodes0 + w.part, cp, 8)) *reinterpret_cast<uint2*>(cp) = code;
    if (kNv || (w.seg & 1) == 0) {
      uint8_t* sp = p.scales[w.part] + row * (p.head_dim / (kNv ? 16 : 32)) +
                    (kNv ? w.seg : w.seg >> 1);
      if (MXFP4_IN_BOUNDS(p, kDbgScales0 + w.part, sp, 1)) *sp = static_cast<uint8_t>(s);
    }
  }
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
  write_status(p);
  const int first = blockIdx.x * p.tokens_per_cta;
  const int avail = p.num_tokens - first;
  const int tokens = avail < p.tokens_per_cta ? avail : p.tokens_per_cta;
  const uint32_t segs = p.head_dim / kElems;
  const uint32_t units = static_cast<uint32_t>(tokens) * 2u * p.num_heads * segs;
  for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
    const Unit w = unit_of(p, first, u, segs);
    const int32_t slot = __ldg(p.slots + w.token);
    uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
    if (slot >= 0 && slot < p.num_slots) {
      const int64_t row = cache_row(p, slot, w.head);
      const uint8_t* cp = p.codes[w.part] + row * (p.head_dim / 2) + w.seg * 8;
      const uint8_t* sp = p.scales[w.part] + row * (p.head_dim / (kNv ? 16 : 32)) +
                          (kNv ? w.seg : w.seg >> 1);
      uint2 c = make_uint2(0u, 0u);
      uint32_t s = 0u;
      if (MXFP4_IN_BOUNDS(p, kDbgCodes0 + w.part, cp, 8) && MXFP4_IN_BOUNDS(p, kDbgScales0 + w.part, sp, 1)) {
        c = ld_stream_v2(cp);
        s = __ldg(sp);
      }
      const bool nan = kNv ? (s & 0x7Fu) == 0x7Fu : s == 255u;
      if (nan) {
        const uint32_t q = kF16 ? 0x7E007E00u : 0x7FC07FC0u;
        o0 = o1 = make_uint4(q, q, q, q);
      } else {
        const float sc = kNv ? e4m3_to_f32(s) : scale_from_e8m0(s);
        const float inv = kNv ? 1.0f / __ldg(p.global_scales[w.part]) : 1.0f;
        o0 = decode8<kNv, kF16>(c.x, sc, inv);
        o1 = decode8<kNv, kF16>(c.y, sc, inv);
      }
    }
    uint8_t* dst = p.out[w.part] +
                   ((static_cast<int64_t>(w.token) * p.num_heads + w.head) * p.head_dim + w.seg * kElems) * 2;
    if (MXFP4_IN_BOUNDS(p, kDbgX0 + w.part, dst, 32)) {
      st_stream_v4(dst, o0);
      st_stream_v4(dst + 16, o1);
    }
  }
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
  // tokens per CTA: about four 16-element units per thread, at least one token
  const int64_t per_token = 2LL * c.num_heads * (c.head_dim / kElems);
  const int64_t t = per_token > 0 ? (4LL * kThreads) / per_token : 1;
  p.tokens_per_cta = static_cast<int32_t>(t < 1 ? 1 : t);
#ifdef MXFP4_DEBUG_BOUNDS
  const int64_t row = static_cast<int64_t>(c.num_heads) * c.head_dim;
  for (int i = 0; i < 2; ++i) {
    debug_range(p.dbg, kDbgCodes0 + i, c.codes[i], p.num_slots * (row / 2));
    debug_range(p.dbg, kDbgScales0 + i, c.scales[i], p.num_slots * (row / (c.nvfp4 ? 16 : 32)));
  }
#endif
  return p;
}

unsigned grid_of(const CacheParams& p) {
  const int64_t g = (static_cast<int64_t>(p.num_tokens) + p.tokens_per_cta - 1) / p.tokens_per_cta;
  return static_cast<unsigned>(g > 0 ? g : 1);  // no tokens: the status word alone
}

}  // namespace

cudaError_t launch_cache_write(const CacheArgs& c, const void* const x[2], int64_t num_tokens,
                               const int64_t token_stride[2], const int64_t head_stride[2],
                               const int32_t* slots, int32_t* status, cudaStream_t stream) {
  CacheParams p = cache_params(c, slots, num_tokens, status);
  for (int i = 0; i < 2; ++i) {
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
  for (int i = 0; i < 2; ++i) {
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

// attention.cu — attention of one query token per sequence over the paged
// 4-bit cache, for sm_103a.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j over the positions j in
//   [max(0, n - window), n) of each sequence, with k and v decoded from
//   MXFP4 (e2m1 * 2^(s-127)) or NVFP4 (e2m1 * e4m3(s) / g).
// One pass over the cache with a running maximum and sum per head, all in
// float32.  A CTA per (sequence, query head); a warp per position, a lane
// per head_dim/32 elements.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 256;

struct AttentionParams {
  const uint8_t* __restrict__ q;
  const uint8_t* __restrict__ codes[2];
  const uint8_t* __restrict__ scales[2];
  const float* __restrict__ global_scales[2];
  const int32_t* __restrict__ page_table;
  const int32_t* __restrict__ seq_lens;
  uint8_t* __restrict__ out;
  float* __restrict__ lse;
  int32_t* __restrict__ status;
  int64_t q_seq_stride;
  int64_t q_head_stride;
  int64_t table_stride;
  int64_t max_len;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_pages;
  int32_t page_size;
  int32_t head_dim;
  int32_t window;
  float softmax_scale;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgQ = 0, kDbgCodes0, kDbgCodes1, kDbgScales0, kDbgScales1, kDbgTable, kDbgOut };

// The positions [lo, hi) of sequence b; a length out of range gives none.
__device__ __forceinline__ bool positions(const AttentionParams& p, int b, int& lo, int& hi) {
  const int n = __ldg(p.seq_lens + b);
  const bool ok = n >= 0 && n <= p.max_len;
  hi = ok ? n : 0;
  lo = p.window > 0 && hi > p.window ? hi - p.window : 0;
  return ok;
}

template <bool kNv>
__device__ __forceinline__ float scale_value(uint32_t s) {
  if constexpr (kNv) return e4m3_to_f32(s);
  return s == 255u ? __uint_as_float(0x7FC00000u) : scale_from_e8m0(s);
}

template <bool kNv, bool kF16>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttentionParams p) {
  __shared__ float s_o[kWarps][kMaxDim];
  __shared__ float s_m[kWarps], s_l[kWarps];
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == static_cast<unsigned>(p.num_seqs * p.num_q_heads)) {  // the status word
    int bad = 0;
    for (int b = warp; b < p.num_seqs; b += kWarps) {
      int lo, hi;
      if (!positions(p, b, lo, hi)) bad = 1;
      const int last = hi > lo ? (hi - 1) / p.page_size : -1;
      for (int i = lo / p.page_size + lane; i <= last; i += 32) {
        const int32_t page = __ldg(p.page_table + b * p.table_stride + i);
        if (page < 0 || page >= p.num_pages) bad = 1;
      }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status = bad ? -7 : 0;
    return;
  }
  const int b = blockIdx.x / p.num_q_heads, h = blockIdx.x % p.num_q_heads;
  const int kvh = h / (p.num_q_heads / p.num_kv_heads);
  const int D = p.head_dim;
  const int per = kNv ? 16 : 32;
  int lo, hi;
  positions(p, b, lo, hi);
  // a lane's elements: pairs 2 * (lane + 32 i)
  float q[8], o[8];
  const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.q) + b * p.q_seq_stride + h * p.q_head_stride;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = (i >> 1) * 64 + lane * 2 + (i & 1);
    o[i] = 0.0f;
    q[i] = 0.0f;
    if (d < D && MXFP4_IN_BOUNDS(p, kDbgQ, qp + d, 2))
      q[i] = kF16 ? __uint_as_float(f16_bits_to_f32_bits(qp[d])) : __uint_as_float(static_cast<uint32_t>(qp[d]) << 16);
  }
  const float kg = kNv ? 1.0f / __ldg(p.global_scales[0]) : 1.0f;
  const float vg = kNv ? 1.0f / __ldg(p.global_scales[1]) : 1.0f;
  float m = -INFINITY, l = 0.0f;
  for (int j = lo + warp; j < hi; j += kWarps) {
    const int32_t page = __ldg(p.page_table + b * p.table_stride + j / p.page_size);
    if (page < 0 || page >= p.num_pages) continue;
    const int64_t row = (static_cast<int64_t>(page) * p.num_kv_heads + kvh) * p.page_size + j % p.page_size;
    float dot = 0.0f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = i * 64 + lane * 2;
      v[2 * i] = v[2 * i + 1] = 0.0f;
      if (d >= D) continue;
      uint32_t h2[2];
      float s[2];
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint8_t* cp = p.codes[part] + row * (D / 2) + d / 2;
        const uint8_t* sp = p.scales[part] + row * (D / per) + d / per;
        h2[part] = 0u;
        s[part] = 0.0f;
        if (MXFP4_IN_BOUNDS(p, kDbgCodes0 + part, cp, 1) && MXFP4_IN_BOUNDS(p, kDbgScales0 + part, sp, 1)) {
          h2[part] = cvt_e2m1x2_to_f16x2(__ldg(cp));
          s[part] = scale_value<kNv>(__ldg(sp));
        }
      }
      dot = fmaf(q[2 * i], half_lo_to_f32(h2[0]) * s[0], dot);
      dot = fmaf(q[2 * i + 1], half_hi_to_f32(h2[0]) * s[0], dot);
      v[2 * i] = half_lo_to_f32(h2[1]) * s[1];
      v[2 * i + 1] = half_hi_to_f32(h2[1]) * s[1];
    }
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
    const float a = dot * kg * p.softmax_scale;
    const float top = fmaxf(m, a);
    const float keep = m == -INFINITY ? 0.0f : expf(m - top);
    const float w = top == -INFINITY ? 0.0f : expf(a - top);
    l = l * keep + w;
    m = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + w * v[i];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = (i >> 1) * 64 + lane * 2 + (i & 1);
    if (d < D) s_o[warp][d] = o[i];
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w)
    if (s_m[w] != -INFINITY) sum += s_l[w] * expf(s_m[w] - top);
  const int64_t head = static_cast<int64_t>(b) * p.num_q_heads + h;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float acc = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (s_m[w] != -INFINITY) acc += s_o[w][d] * expf(s_m[w] - top);
    acc = sum > 0.0f || sum != sum ? acc * vg / sum : 0.0f;
    uint16_t* y = reinterpret_cast<uint16_t*>(p.out) + head * D + d;
    if (MXFP4_IN_BOUNDS(p, kDbgOut, y, 2))
      *y = kF16 ? __half_as_ushort(__float2half_rn(acc)) : static_cast<uint16_t>(cvt_bf16x2(acc, 0.0f));
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[head] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

int64_t attention_workspace_floats(int64_t, int32_t, int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t stream) {
  const CacheArgs& c = a.cache;
  AttentionParams p{};
  p.q = static_cast<const uint8_t*>(a.q);
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = c.codes[i];
    p.scales[i] = c.scales[i];
    p.global_scales[i] = c.global_scales[i];
  }
  p.page_table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.out = static_cast<uint8_t*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.q_seq_stride = a.q_seq_stride;
  p.q_head_stride = a.q_head_stride;
  p.table_stride = a.table_stride;
  p.max_len = a.max_pages * c.page_size;
  p.num_seqs = static_cast<int32_t>(a.num_seqs);
  p.num_q_heads = c.head_dim > 0 ? a.num_q_heads : 0;
  p.num_kv_heads = c.num_heads;
  p.num_pages = static_cast<int32_t>(c.num_pages);
  p.page_size = c.page_size;
  p.head_dim = c.head_dim;
  p.window = a.window;
  p.softmax_scale = a.softmax_scale;
#ifdef MXFP4_DEBUG_BOUNDS
  const int64_t rows = c.num_pages * c.page_size * c.num_heads;
  debug_range(p.dbg, kDbgQ, a.q, a.num_seqs > 0 && a.num_q_heads > 0
      ? ((a.num_seqs - 1) * a.q_seq_stride + (a.num_q_heads - 1) * a.q_head_stride + c.head_dim) * 2 : 0);
  for (int i = 0; i < 2; ++i) {
    debug_range(p.dbg, kDbgCodes0 + i, c.codes[i], rows * (c.head_dim / 2));
    debug_range(p.dbg, kDbgScales0 + i, c.scales[i], rows * (c.head_dim / (c.nvfp4 ? 16 : 32)));
  }
  debug_range(p.dbg, kDbgOut, a.out, a.num_seqs * a.num_q_heads * c.head_dim * 2);
#endif
  const unsigned grid = static_cast<unsigned>(p.num_seqs) * p.num_q_heads + (a.status ? 1 : 0);
  if (grid == 0) return cudaSuccess;
  const auto kernel = c.nvfp4 ? (c.f16 ? attention_kernel<true, true> : attention_kernel<true, false>)
                              : (c.f16 ? attention_kernel<false, true> : attention_kernel<false, false>);
  return launch_pdl(kernel, grid, kThreads, 0, stream, p);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_attention() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

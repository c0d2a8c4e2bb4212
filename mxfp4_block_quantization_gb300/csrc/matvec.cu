// matvec.cu — products of a few tokens with 4-bit weights (MXFP4 or NVFP4),
// dense and per expert segment, for sm_103a.
//
//   y[r, n] = sum_k x[r, k] * W[n, k]
//   MXFP4: W = e2m1(code) * 2^(s-127), one scale byte per 32 elements of K
//   NVFP4: W = e2m1(code) * e4m3(s) / g, one scale byte per 16 elements
// Sums are float32; the result is rounded once to the output's type.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"

namespace mxfp4 {
namespace {

struct MatvecParams {
  const uint8_t* __restrict__ x;
  const int32_t* __restrict__ row_index;
  const int32_t* __restrict__ offsets;
  const uint8_t* __restrict__ codes;
  const uint8_t* __restrict__ scales;
  const float* __restrict__ global_scales;
  uint8_t* __restrict__ y;
  int32_t* __restrict__ status;
  int64_t src_rows;
  int64_t ldx;
  int64_t ldy;
  int64_t rows;
  int64_t N;
  int64_t expert_codes;   // bytes of one expert's codes
  int64_t expert_scales;  // bytes of one expert's tiled scales
  int32_t K;
  int32_t E;
  int32_t nKT;  // 4-column scale chunks of a row
  int32_t y_f32;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgX = 0, kDbgCodes, kDbgScales, kDbgGlobal, kDbgY, kDbgIndex, kDbgOffsets };

template <bool kNv>
__device__ __forceinline__ float scale_value(uint32_t s) {
  if constexpr (kNv) {
    return e4m3_to_f32(s);
  } else {
    return s == 255u ? __uint_as_float(0x7FC00000u) : scale_from_e8m0(s);
  }
}

template <bool kF16>
__device__ __forceinline__ float value16(uint16_t v) {
  return kF16 ? __uint_as_float(f16_bits_to_f32_bits(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Whether the expert offsets are 0 = o[0] <= ... <= o[E] <= rows, by the whole
// CTA.
__device__ __forceinline__ bool offsets_ok(const MatvecParams& p) {
  int bad = 0;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    const int32_t o = __ldg(p.offsets + e);
    if (e == 0 ? o != 0 : o < __ldg(p.offsets + e - 1)) bad = 1;
    if (o < 0 || o > p.rows) bad = 1;
  }
  return __syncthreads_or(bad) == 0;
}

template <bool kNv, bool kF16>
__global__ void __launch_bounds__(256) matvec_kernel(const MatvecParams p) {
  constexpr int kBlk = kNv ? 16 : 32;
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.offsets != nullptr) {
    const bool ok = offsets_ok(p);
    if (blockIdx.x == 0 && blockIdx.y == 0 && p.status != nullptr) {
      int bad = 0;
      if (ok && p.row_index != nullptr)
        for (int r = threadIdx.x; r < __ldg(p.offsets + p.E); r += blockDim.x) {
          const int32_t i = __ldg(p.row_index + r);
          if (i < 0 || i >= p.src_rows) bad = 1;
        }
      bad = __syncthreads_or(bad);
      if (threadIdx.x == 0) *p.status = !ok ? -6 : bad ? -7 : 0;
    }
    if (!ok) return;
  }
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (n >= p.N) return;
  for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
    int e = 0;
    int64_t src = r;
    if (p.offsets != nullptr) {
      if (r >= __ldg(p.offsets + p.E)) return;
      e = find_segment(p.offsets, p.E, static_cast<int>(r), __ldg(p.offsets + p.E));
      if (p.row_index != nullptr) src = __ldg(p.row_index + r);
    }
    const bool live = src >= 0 && src < p.src_rows;
    const uint8_t* codes = p.codes + e * p.expert_codes + n * (p.K / 2);
    const uint8_t* scales = p.scales + e * p.expert_scales + (n / 128) * p.nKT * kChunkBytes +
                            (n % 32) * 16 + (n % 128) / 32 * 4;
    float acc = 0.0f;
    if (live) {
      const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + src * p.ldx;
      for (int k = lane * 2; k < p.K; k += 64) {
        const int c = k / kBlk;
        const uint8_t* sp = scales + static_cast<int64_t>(c >> 2) * kChunkBytes + (c & 3);
        if (!MXFP4_IN_BOUNDS(p, kDbgX, x + k, 4) || !MXFP4_IN_BOUNDS(p, kDbgCodes, codes + k / 2, 1) ||
            !MXFP4_IN_BOUNDS(p, kDbgScales, sp, 1))
          continue;
        const uint32_t h = cvt_e2m1x2_to_f16x2(__ldg(codes + k / 2));
        const float s = scale_value<kNv>(__ldg(sp));
        acc = fmaf(value16<kF16>(x[k]) * half_lo_to_f32(h), s, acc);
        acc = fmaf(value16<kF16>(x[k + 1]) * half_hi_to_f32(h), s, acc);
      }
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    if (kNv && p.K > 0 && MXFP4_IN_BOUNDS(p, kDbgGlobal, p.global_scales + e, 4))
      acc /= __ldg(p.global_scales + e);
    if (lane == 0) {
      if (p.y_f32) {
        float* y = reinterpret_cast<float*>(p.y) + r * p.ldy + n;
        if (MXFP4_IN_BOUNDS(p, kDbgY, y, 4)) *y = acc;
      } else {
        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + r * p.ldy + n;
        if (MXFP4_IN_BOUNDS(p, kDbgY, y, 2))
          *y = kF16 ? __half_as_ushort(__float2half_rn(acc)) : static_cast<uint16_t>(cvt_bf16x2(acc, 0.0f));
      }
    }
  }
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t stream) {
  MatvecParams p{};
  p.x = static_cast<const uint8_t*>(a.x);
  p.row_index = a.row_index;
  p.offsets = a.offsets;
  p.codes = a.codes;
  p.scales = a.scales;
  p.global_scales = a.global_scales;
  p.y = static_cast<uint8_t*>(a.y);
  p.status = a.status;
  p.src_rows = a.src_rows;
  p.ldx = a.ldx;
  p.ldy = a.ldy;
  p.rows = a.rows;
  p.N = a.N;
  p.K = static_cast<int32_t>(a.K);
  p.E = a.E;
  p.nKT = static_cast<int32_t>((a.K / (a.nvfp4 ? 16 : 32) + 3) / 4);
  p.expert_codes = a.N * (a.K / 2);
  p.expert_scales = (a.N + 127) / 128 * p.nKT * kChunkBytes;
  p.y_f32 = a.y_f32;
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.dbg, kDbgX, a.x, a.src_rows > 0 ? ((a.src_rows - 1) * a.ldx + a.K) * 2 : 0);
  debug_range(p.dbg, kDbgCodes, a.codes, a.E * p.expert_codes);
  debug_range(p.dbg, kDbgScales, a.scales, a.E * p.expert_scales);
  debug_range(p.dbg, kDbgGlobal, a.global_scales, a.nvfp4 ? a.E * 4 : 0);
  debug_range(p.dbg, kDbgY, a.y, a.rows > 0 ? ((a.rows - 1) * a.ldy + a.N) * (a.y_f32 ? 4 : 2) : 0);
#endif
  cudaLaunchConfig_t cfg = {};
  const int64_t tiles = (a.N + 7) / 8;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles > 0 ? tiles : 1),
                     static_cast<unsigned>(a.rows > 32768 ? 32768 : a.rows > 0 ? a.rows : 1));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = a.nvfp4 ? (a.f16 ? matvec_kernel<true, true> : matvec_kernel<true, false>)
                              : (a.f16 ? matvec_kernel<false, true> : matvec_kernel<false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_matvec() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

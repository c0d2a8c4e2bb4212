// gemm.cu — products of 4-bit activations with 4-bit weights for sm_103a, the
// simple form: a CTA of 256 threads makes 64 rows by 64 columns of y, both
// operands decoded to float32 in shared memory 32 elements of K at a time.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "../../include/mxfp4.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kSide = 64;

struct GemmParams {
  GemmArgs a;
  int64_t expert_codes;
  int64_t expert_scales;
  int nKT;
  int cols;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};
enum : int { kDbgXCodes = 0, kDbgXScales, kDbgCodes, kDbgScales, kDbgOffsets, kDbgResidual, kDbgY, kDbgStatus };

__device__ __forceinline__ float load_half(const void* p, int64_t i, bool f16) {
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return f16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ float activate(float z, int act) {
  if (act == MXFP4_ACT_SILU) return z / (1.0f + expf(-z));
  if (act == MXFP4_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  if (act == MXFP4_ACT_GELU_TANH)
    return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
  return z;
}

// Element k of a row whose scales begin at tiled row r.
__device__ float element(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t r, int k,
                         int K, int nKT, bool nvfp4) {
  const uint32_t b = codes[row * (K / 2) + k / 2];
  const uint32_t h2 = cvt_e2m1x2_to_f16x2(b);
  const float v = k & 1 ? half_hi_to_f32(h2) : half_lo_to_f32(h2);
  const int c = k / (nvfp4 ? 16 : 32);
  const uint32_t s = scales[((r / 128) * nKT + c / 4) * 512 + chunk_offset(static_cast<int>(r % 128), c % 4)];
  if (nvfp4) return v * e4m3_to_f32(s);
  return s == 255u ? NAN : v * scale_from_e8m0(s);
}

__global__ void __launch_bounds__(kThreads) gemm_kernel(const GemmParams p) {
  __shared__ float xs[kSide][33], ws[2][kSide][33];
  __shared__ int s_bad, s_pad;
  pdl_wait();
  pdl_release();
  const GemmArgs& a = p.a;
  const int e = blockIdx.z;
  int64_t lo = 0, hi = a.rows, pad = 0;
  if (threadIdx.x == 0) s_bad = 0, s_pad = 0;
  __syncthreads();
  if (a.offsets) {
    int bad = threadIdx.x == 0 && a.offsets[0] != 0, sum = 0;
    for (int i = threadIdx.x; i < a.E; i += kThreads) {
      const int from = a.offsets[i], to = a.offsets[i + 1];
      bad |= from > to || from < 0 || to > a.rows;
      if (i < e) sum += (to - from + 127) / 128 * 128;
    }
    if (bad) atomicOr(&s_bad, 1);
    atomicAdd(&s_pad, sum);
    __syncthreads();
    if (a.status && blockIdx.x == 0 && e == 0 && threadIdx.x == 0)
      *a.status = s_bad ? MXFP4_EOFFSETS : MXFP4_OK;
    if (s_bad || a.E == 0 || p.cols == 0) return;
    lo = a.offsets[e], hi = a.offsets[e + 1], pad = s_pad;
  }
  const bool gated = a.gate != MXFP4_GATE_NONE;
  const int n0 = blockIdx.x * kSide;
  const int first = a.gate == MXFP4_GATE_SECOND ? p.cols : 0;   // the activated rows of W
  const int other = a.gate == MXFP4_GATE_SECOND ? 0 : p.cols;
  const uint8_t* const wc = a.codes + e * p.expert_codes;
  const uint8_t* const wsc = a.scales + e * p.expert_scales;
  const float alpha = a.nvfp4 && a.K > 0 ? (1.0f / a.x_globals[e]) * (1.0f / a.globals[e]) : 1.0f;
  const int K = static_cast<int>(a.K);
  for (int64_t t0 = lo; t0 < hi; t0 += kSide) {
    float acc[2][4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < kSide * 32; i += kThreads) {
        const int r = i / 32, k = i % 32;
        xs[r][k] = t0 + r < hi ? element(a.x_codes, a.x_scales, t0 + r, pad + t0 - lo + r, k0 + k, K, p.nKT, a.nvfp4) : 0.0f;
        const bool in = n0 + r < p.cols;
        ws[0][r][k] = in ? element(wc, wsc, first + n0 + r, first + n0 + r, k0 + k, K, p.nKT, a.nvfp4) : 0.0f;
        if (gated) ws[1][r][k] = in ? element(wc, wsc, other + n0 + r, other + n0 + r, k0 + k, K, p.nKT, a.nvfp4) : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) {
            const float x = xs[threadIdx.x / 16 + 16 * i][k];
            acc[0][i][j] = fmaf(x, ws[0][threadIdx.x % 16 + 16 * j][k], acc[0][i][j]);
            if (gated) acc[1][i][j] = fmaf(x, ws[1][threadIdx.x % 16 + 16 * j][k], acc[1][i][j]);
          }
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + threadIdx.x / 16 + 16 * i;
        const int n = n0 + threadIdx.x % 16 + 16 * j;
        if (t >= hi || n >= p.cols) continue;
        float z = acc[0][i][j] * alpha, u = acc[1][i][j] * alpha;
        if (a.bias) z += load_half(a.bias, e * a.N + first + n, a.f16);
        if (a.bias && gated) u += load_half(a.bias, e * a.N + other + n, a.f16);
        float y = activate(z, a.activation);
        if (gated) y *= u;
        if (a.residual) y += load_half(a.residual, t * a.ldr + n, a.f16);
        static_cast<uint16_t*>(a.y)[t * a.ldy + n] =
            a.f16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
      }
  }
}

}  // namespace

cudaError_t launch_gemm(const GemmArgs& a, cudaStream_t stream) {
  GemmParams p{};
  p.a = a;
  p.nKT = static_cast<int>((a.K / (a.nvfp4 ? 16 : 32) + 3) / 4);
  p.cols = static_cast<int>(a.gate != MXFP4_GATE_NONE ? a.N / 2 : a.N);
  p.expert_codes = a.N * (a.K / 2);
  p.expert_scales = (a.N + 127) / 128 * p.nKT * kChunkBytes;
  const dim3 grid(p.cols > 0 ? (p.cols + kSide - 1) / kSide : 1, 1, a.E > 0 ? a.E : 1);
  return launch_pdl(gemm_kernel, grid, kThreads, 0, stream, p);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_gemm() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

// combine.cu — the experts' rows back to their tokens, for sm_103a:
//   y[t] = residual[t] + sum_j weights[t, j] * rows[dest_rows[t, j]].
//
// Bandwidth bounds it: every dispatched row is read once.  A thread has eight
// consecutive columns of a token (one where rows are not in whole 16-byte
// pieces) and adds the routes in order, the rows of up to kAhead of them in
// flight; nothing is shared between threads, so equal calls give equal bits.
// 16384 tokens of 8 rows of 7168 and a residual take 358 us: 6.3 TB/s, 93 % of the
// measured copy rate.  Of 1024 columns 45 us (the copy rate), of 256 9.1, of 64 3.9; but
// the status word's CTA takes 12 to 14 us over those 131072 entries, whatever the rows'
// length.  Of 2047 columns, one to a thread, 290 us (floor 89).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "../../include/mxfp4.h"

namespace mxfp4 {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kAhead = 4;  // routes whose rows are loaded before they are added

struct CombineParams {
  const uint8_t* rows;
  const int32_t* dest;
  const float* weights;
  const uint8_t* residual;  // or NULL
  uint8_t* y;
  int32_t* status;          // or NULL
  int64_t total_rows;
  int64_t ldr;
  int64_t ld_res;
  int64_t ldy;
  int32_t tokens;
  int32_t top_k;
  int32_t N;
  int32_t chunks;           // of a row, a thread each
  int32_t row_blocks;       // CTAs to a row, or
  int32_t block_rows;       // rows to a CTA
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgRows = 0, kDbgDest, kDbgWeights, kDbgResidual, kDbgY, kDbgStatus };

template <bool kF16>
__device__ __forceinline__ float widen(uint16_t v) {
  if constexpr (kF16) return __half2float(__ushort_as_half(v));
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <bool kF16>
__device__ __forceinline__ uint16_t narrow(float v) {
  if constexpr (kF16) return __half_as_ushort(__float2half_rn(v));
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
template <bool kF16>
__device__ __forceinline__ void widen2(uint32_t v, float* f) {
  f[0] = widen<kF16>(static_cast<uint16_t>(v));
  f[1] = widen<kF16>(static_cast<uint16_t>(v >> 16));
}

// A chunk of a row: kCols elements as they lie.
template <bool kF32, int kCols>
struct Piece {
  static constexpr int kBytes = kCols * (kF32 ? 4 : 2);
  uint4 v[kBytes >= 16 ? kBytes / 16 : 1];
};

template <bool kF32, int kCols>
__device__ __forceinline__ void load_piece(const CombineParams& p, int slot, const uint8_t* at,
                                           Piece<kF32, kCols>& out) {
  if constexpr (kCols == 8) {
#pragma unroll
    for (int i = 0; i < Piece<kF32, kCols>::kBytes / 16; ++i)
      out.v[i] = MXFP4_IN_BOUNDS(p, slot, at + 16 * i, 16) ? ld_stream_v4(at + 16 * i)
                                                           : make_uint4(0u, 0u, 0u, 0u);
  } else if constexpr (kF32) {
    out.v[0].x = MXFP4_IN_BOUNDS(p, slot, at, 4) ? __ldg(reinterpret_cast<const uint32_t*>(at)) : 0u;
  } else {
    out.v[0].x = MXFP4_IN_BOUNDS(p, slot, at, 2) ? __ldg(reinterpret_cast<const uint16_t*>(at)) : 0u;
  }
}
template <bool kF32, int kCols, bool kF16>
__device__ __forceinline__ void values_of(const Piece<kF32, kCols>& piece, float (&f)[kCols]) {
  if constexpr (kCols == 8 && kF32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(piece.v[i].x), f[4 * i + 1] = __uint_as_float(piece.v[i].y);
      f[4 * i + 2] = __uint_as_float(piece.v[i].z), f[4 * i + 3] = __uint_as_float(piece.v[i].w);
    }
  } else if constexpr (kCols == 8) {
    widen2<kF16>(piece.v[0].x, f);
    widen2<kF16>(piece.v[0].y, f + 2);
    widen2<kF16>(piece.v[0].z, f + 4);
    widen2<kF16>(piece.v[0].w, f + 6);
  } else if constexpr (kF32) {
    f[0] = __uint_as_float(piece.v[0].x);
  } else {
    f[0] = widen<kF16>(static_cast<uint16_t>(piece.v[0].x));
  }
}

// The status word, by a CTA of its own: any entry outside [-1, total_rows).
__device__ void check_entries(const CombineParams& p) {
  const int64_t n = static_cast<int64_t>(p.tokens) * p.top_k;
  int bad = 0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    if (!MXFP4_IN_BOUNDS(p, kDbgDest, p.dest + i, 4)) continue;
    const int32_t r = __ldg(p.dest + i);
    bad |= r < -1 || r >= p.total_rows;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && MXFP4_IN_BOUNDS(p, kDbgStatus, p.status, 4))
    *p.status = bad ? MXFP4_EINDEX : MXFP4_OK;
}

template <bool kF32, bool kF16, int kCols>
__global__ void __launch_bounds__(kMaxThreads) moe_combine_kernel(const CombineParams p) {
  pdl_wait();
  pdl_release();
  int block = blockIdx.x;
  if (p.status != nullptr) {
    if (block == 0) {
      check_entries(p);
      return;
    }
    --block;
  }
  int t, chunk;
  if (p.block_rows > 1) {
    const int local = threadIdx.x / p.chunks;
    t = block * p.block_rows + local;
    chunk = threadIdx.x - local * p.chunks;
    if (local >= p.block_rows) return;
  } else {
    t = block / p.row_blocks;
    chunk = (block - t * p.row_blocks) * blockDim.x + threadIdx.x;
  }
  if (t >= p.tokens || chunk >= p.chunks) return;
  const int64_t col = static_cast<int64_t>(chunk) * kCols;
  constexpr int kSize = kF32 ? 4 : 2;

  float sum[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) sum[c] = 0.0f;
  if (p.residual != nullptr) {
    Piece<false, kCols> r;
    const uint8_t* const at = p.residual + (t * p.ld_res + col) * 2;  // may be y: a plain load
    if constexpr (kCols == 8)
      r.v[0] = MXFP4_IN_BOUNDS(p, kDbgResidual, at, 16) ? *reinterpret_cast<const uint4*>(at)
                                                        : make_uint4(0u, 0u, 0u, 0u);
    else
      r.v[0].x = MXFP4_IN_BOUNDS(p, kDbgResidual, at, 2) ? *reinterpret_cast<const uint16_t*>(at) : 0u;
    values_of<false, kCols, kF16>(r, sum);
  }
  const int64_t routes = static_cast<int64_t>(t) * p.top_k;
  for (int j0 = 0; j0 < p.top_k; j0 += kAhead) {
    int32_t row[kAhead];
    float w[kAhead];
    Piece<kF32, kCols> piece[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t at = routes + j0 + j;
      row[j] = j0 + j < p.top_k && MXFP4_IN_BOUNDS(p, kDbgDest, p.dest + at, 4)
                   ? __ldg(p.dest + at) : -1;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (row[j] >= 0 && row[j] < p.total_rows) {
        const int64_t at = routes + j0 + j;
        w[j] = MXFP4_IN_BOUNDS(p, kDbgWeights, p.weights + at, 4) ? __ldg(p.weights + at) : 0.0f;
        load_piece<kF32, kCols>(p, kDbgRows, p.rows + (row[j] * p.ldr + col) * kSize, piece[j]);
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (row[j] >= 0 && row[j] < p.total_rows) {
        float f[kCols];
        values_of<kF32, kCols, kF16>(piece[j], f);
#pragma unroll
        for (int c = 0; c < kCols; ++c) sum[c] = fmaf(w[j], f[c], sum[c]);
      }
  }
  uint8_t* const out = p.y + (t * p.ldy + col) * 2;
  if constexpr (kCols == 8) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = narrow<kF16>(sum[2 * i]) | static_cast<uint32_t>(narrow<kF16>(sum[2 * i + 1])) << 16;
    if (MXFP4_IN_BOUNDS(p, kDbgY, out, 16)) st_stream_v4(out, make_uint4(v[0], v[1], v[2], v[3]));
  } else {
    if (MXFP4_IN_BOUNDS(p, kDbgY, out, 2)) *reinterpret_cast<uint16_t*>(out) = narrow<kF16>(sum[0]);
  }
}

template <bool kF32, bool kF16>
cudaError_t launch_typed(CombineParams& p, bool wide, cudaStream_t stream) {
  p.chunks = wide ? p.N / 8 : p.N > 0 ? p.N : 1;
  p.block_rows = p.chunks < kMaxThreads ? kMaxThreads / p.chunks : 1;
  p.row_blocks = (p.chunks + kMaxThreads - 1) / kMaxThreads;
  // a row's chunks in even parts of whole warps
  const int threads = p.block_rows > 1 ? kMaxThreads
                                       : ((p.chunks + p.row_blocks - 1) / p.row_blocks + 31) / 32 * 32;
  int64_t blocks = p.block_rows > 1 ? (p.tokens + p.block_rows - 1) / p.block_rows
                                    : static_cast<int64_t>(p.tokens) * p.row_blocks;
  if (p.N == 0) blocks = 0;  // the status word alone
  blocks += p.status != nullptr ? 1 : 0;
  if (blocks == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(blocks));
  return wide ? launch_pdl(moe_combine_kernel<kF32, kF16, 8>, grid, threads, 0, stream, p)
              : launch_pdl(moe_combine_kernel<kF32, kF16, 1>, grid, threads, 0, stream, p);
}

bool pieces(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

}  // namespace

cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t stream) {
  CombineParams p{};
  p.rows = static_cast<const uint8_t*>(a.rows);
  p.dest = a.dest;
  p.weights = a.weights;
  p.residual = static_cast<const uint8_t*>(a.residual);
  p.y = static_cast<uint8_t*>(a.y);
  p.status = a.status;
  p.total_rows = a.total_rows;
  p.ldr = a.ldr;
  p.ld_res = a.ld_res;
  p.ldy = a.ldy;
  p.tokens = static_cast<int32_t>(a.num_tokens);
  p.top_k = a.top_k;
  p.N = static_cast<int32_t>(a.N);
  const int size = a.rows_f32 ? 4 : 2;
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.dbg, kDbgRows, a.rows, a.total_rows > 0 ? ((a.total_rows - 1) * a.ldr + a.N) * size : 0);
  debug_range(p.dbg, kDbgDest, a.dest, a.num_tokens * a.top_k * 4);
  debug_range(p.dbg, kDbgWeights, a.weights, a.num_tokens * a.top_k * 4);
  debug_range(p.dbg, kDbgResidual, a.residual, a.residual ? ((a.num_tokens - 1) * a.ld_res + a.N) * 2 : 0);
  debug_range(p.dbg, kDbgY, a.y, a.num_tokens > 0 ? ((a.num_tokens - 1) * a.ldy + a.N) * 2 : 0);
  debug_range(p.dbg, kDbgStatus, a.status, a.status ? 4 : 0);
#endif
  // eight columns to a thread where every row is in 16-byte pieces
  const bool wide = p.N > 0 && p.N % 8 == 0 && pieces(a.rows, a.ldr, size) && pieces(a.y, a.ldy, 2) &&
                    (a.residual == nullptr || pieces(a.residual, a.ld_res, 2));
  if (a.rows_f32)
    return a.f16 ? launch_typed<true, true>(p, wide, stream) : launch_typed<true, false>(p, wide, stream);
  return a.f16 ? launch_typed<false, true>(p, wide, stream) : launch_typed<false, false>(p, wide, stream);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_combine() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

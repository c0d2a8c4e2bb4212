// gemm.cu — products of 4-bit activations with 4-bit weights for sm_103a, dense
// and per expert, with bias, activation, gate and residual in the epilogue
// (formulas in include/mxfp4.h).
//
// The codes and tiled scales go to the tensor cores as they lie: a block-scaled
// tcgen05.mma takes E2M1 operands packed two to a byte and, of each 512-byte
// chunk of the 128x4-tiled scales, the copy to tensor memory that tcgen05.cp
// makes.  Nothing is decoded.
//
// The 128-row operand is always the weights, tokens are the columns: their
// number in an instruction is any multiple of 16 up to 256, so one kernel serves
// one token and many.  A CTA's tile is 128 rows of the weights by 256 tokens, or,
// with a gate, 128 rows of each half by 128 tokens, whose two sums meet in the
// epilogue.  256 elements of K at a time (a stage) are 16 KB for each 128 rows.
//
// Warp 0 copies stages ahead (TMA, a ring of four to eight), one thread of warp 1 issues
// the scales' copies and the products, warp 2 mends scales where a half of gated
// weights or K end inside of their tiles, warp 3 finds the tiles, warps 4 to 19 take
// the sums from tensor
// memory into registers, which frees it for the next tile, and finish them.  Each
// CTA walks every gridDim-th tile.  Where tiles are few, a cluster of up to 8 CTAs
// shares a tile, each with a part of K, and adds the parts in rank order through
// distributed shared memory: equal calls give equal bits.
//
// Measured (calls in a graph): 4096 tokens by 7168 x 7168 MXFP4 66.5 us (6.3 PFLOP/s): to
// each CTA's six tiles 28 stages of 0.33 us, where a stage's four products take 0.26, for
// the copies, and 1.8 us to a tile for its turn (by the times of K = 2048 to 10240).  With
// bias and residual 77 us (5.5 PFLOP/s): the epilogue of a tile then takes 8 us (the call
// with K = 512 48 us, without a residual 16), which the next tile's products hide but for
// 1.7.  128 experts' gated 1536 x 2048 by 16384 tokens' 8 routes 171 us (4.8 PFLOP/s; 187
// between calls on other inputs): 4.3 us to a tile, of which its 8 stages 2.7 and the rest
// its turn.  The same by 64 tokens' 8 routes 36 us: HBM, 5.8 TB/s.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fragments.cuh"
#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "tensor_core.cuh"
#include "../../include/mxfp4.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 640;
constexpr int kFirstEpilogue = 4;              // warp
constexpr int kEpilogueWarps = 16;
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 224 * 1024;
constexpr int kRows = 128;                     // of an operand's tile
constexpr int kStageBytes = 128;               // of a row's codes: 256 elements
constexpr int kSlab = kRows * kStageBytes;     // 16 KB
constexpr int kSteps = 4;                      // products of 64 elements to a stage
constexpr int kColumns = 512;
constexpr int kJobs = 4;                       // tiles found ahead
// tensor memory, all of which a CTA has (so that it begins at column 0): sums, then
// the scales of both weight tiles and of the tokens
constexpr uint32_t kSecond = 128;              // sums of the other 128 tokens, or of the second half
constexpr uint32_t kScalesA = 256, kScalesB = 288;

// A stage's scales of 128 rows: two chunks of 512 bytes (four with NVFP4), for
// three tiles and, where the second half of gated weights does not begin at a
// tile of the scales, the tile behind it.  Before them are the codes: one or two
// tiles of weights, and the tokens.
template <bool kNv>
struct Layout {
  static constexpr int kChunks = kNv ? 4 : 2;
  static constexpr int kScales = kChunks * 512;
};

struct GemmMore {
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

struct GemmParams {
  const uint8_t* x_scales;
  const uint8_t* scales;
  const float* x_globals;
  const float* globals;
  const int32_t* offsets;   // NULL: dense
  const uint16_t* bias;     // or NULL
  const uint16_t* residual; // or NULL
  uint16_t* y;
  int32_t* status;          // or NULL
  int64_t expert_scales;    // bytes of one expert's tiled scales
  int64_t ldr;
  int64_t ldy;
  int32_t rows;
  int32_t N;
  int32_t cols;             // of y
  int32_t E;
  int32_t nKT;              // scale chunks of a row
  int32_t steps;            // products along K
  int32_t stages;           // stages along K
  int32_t blocks;           // scales of a row
  int32_t row_tiles;        // tiles of the weights' rows
  int32_t box_rows;         // tokens' rows to a copy
  int32_t tile_tokens;      // tokens of a tile at most
  uint32_t ring_stages;
  uint32_t stage_bytes;     // of which the scales' begin at
  uint32_t scales_at;
  int32_t activation;
  bool gate_second;
  bool paired;              // rows of y lie in whole words
  bool paired_residual;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
  GemmMore more;
};

// Bounds build: which role of the last CTA takes no step in its first tile, so that the
// others' waits for it run out.
enum : int { kStallNone = 0, kStallTiles, kStallCopies, kStallProducts };
#ifdef MXFP4_DEBUG_BOUNDS
__device__ int g_debug_stall;
__device__ __forceinline__ bool stalled(int role) {
  return *const_cast<volatile int*>(&g_debug_stall) == role && blockIdx.x == gridDim.x - 1;
}
#else
__device__ __forceinline__ bool stalled(int) { return false; }
#endif

enum : int { kDbgXScales = 0, kDbgScales, kDbgOffsets, kDbgBias, kDbgResidual, kDbgY, kDbgStatus, kDbgXGlobals };
enum : int { kDbgGlobals = 0 };

__device__ __forceinline__ int32_t offset_at(const GemmParams& p, int e) {
  const int32_t* at = p.offsets + e;
  return MXFP4_IN_BOUNDS(p, kDbgOffsets, at, 4) ? __ldg(at) : 0;
}

// A tile: tokens [row, row + n) of expert e, whose scales begin at tiled row
// `padded`, by weight rows from r0 on (of each half).
struct Tile {
  int e, row, n, padded, r0;
};

// A tile as warp 3 hands it to the others (n < 0: there are no more), with the row
// of its weights and where its scales begin: of the weights (both halves' tiles), of
// the tokens.
struct Job {
  Tile t;
  int w_row;
  int64_t scales, upper, x_scales;
};

// The tiles in order of expert, weight rows, tokens.  A warp finds them
// together, 32 experts at a time; its lanes agree.
struct Walk {
  int e0 = -32, before = 0, padded_before = 0;  // of the experts below e0
  int lo = 0, n = 0, tiles = 0, sum = 0, padded = 0;  // the lane's expert: sum up to and with it
  int block_tiles = 0, block_padded = 0;

  __device__ bool find(const GemmParams& p, int index, Tile& t) {
    const int lane = threadIdx.x & 31;
    if (p.offsets == nullptr) {
      const int token_tiles = (p.rows + p.tile_tokens - 1) / p.tile_tokens;
      const int r = index / token_tiles, c = index - r * token_tiles;
      if (r >= p.row_tiles) return false;
      t = Tile{0, c * p.tile_tokens, min(p.tile_tokens, p.rows - c * p.tile_tokens), c * p.tile_tokens, r * kRows};
      return true;
    }
    while (index >= before + block_tiles) {
      before += block_tiles, padded_before += block_padded;
      e0 += 32;
      if (e0 >= p.E) return false;
      const int e = e0 + lane;
      n = 0;
      if (e < p.E) lo = offset_at(p, e), n = offset_at(p, e + 1) - lo;
      tiles = (n + p.tile_tokens - 1) / p.tile_tokens * p.row_tiles;
      padded = (n + kRows - 1) / kRows * kRows;
      sum = tiles;
      int psum = padded;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, sum, d), b = __shfl_up_sync(0xFFFFFFFFu, psum, d);
        if (lane >= d) sum += a, psum += b;
      }
      block_tiles = __shfl_sync(0xFFFFFFFFu, sum, 31);
      block_padded = __shfl_sync(0xFFFFFFFFu, psum, 31);
      padded = psum - padded;
    }
    const int l = __ffs(__ballot_sync(0xFFFFFFFFu, index < before + sum)) - 1;
    const int rows = __shfl_sync(0xFFFFFFFFu, n, l);
    const int first = before + __shfl_sync(0xFFFFFFFFu, sum - tiles, l);
    const int token_tiles = (rows + p.tile_tokens - 1) / p.tile_tokens;
    const int r = (index - first) / token_tiles, c = index - first - r * token_tiles;
    t = Tile{e0 + l, __shfl_sync(0xFFFFFFFFu, lo, l) + c * p.tile_tokens, min(p.tile_tokens, rows - c * p.tile_tokens),
             padded_before + __shfl_sync(0xFFFFFFFFu, padded, l) + c * p.tile_tokens, r * kRows};
    return true;
  }
};

struct Barriers {
  uint64_t full[kMaxStages], mended[kMaxStages], empty[kMaxStages], sums_full, sums_empty, job_full[kJobs], job_empty[kJobs], drained;
  Job job[kJobs];
  uint32_t columns;  // tensor memory's address
  uint32_t gave_up;
};

// --------------------------------------------------------------- epilogue
template <bool kF16>
__device__ __forceinline__ float widen(uint16_t v) {
  return kF16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}
// Two values as halves of y's type, `lo` in the low half.
template <bool kF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return kF16 ? pack_f16x2(lo, hi) : cvt_bf16x2(lo, hi);
}

// The fast exponential (of 2: 2^-22 off; of e: and 2^-23 |x| for the argument's product
// with log2 e) and inverse (2^-23), results below 2^-126 as 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_exp(float x) { return fast_exp2(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// z / (1 + e^-u), off by 2^-21 and 2^-23 |u| of itself (2^-16 at u = -88, past which it
// is 0), which a later rounding to 16 bits hides.
__device__ __forceinline__ float sigmoid_times(float z, float u) { return z * fast_inverse(1.0f + fast_exp(-u)); }
template <int kCount>
__device__ __forceinline__ void activate(float (&z)[kCount], int act) {
  if (act == MXFP4_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) z[j] = sigmoid_times(z[j], z[j]);
  } else if (act == MXFP4_ACT_GELU) {
    // max(z, 0) - |z| erfc(x) / 2, x = |z| / sqrt(2).  erfc(x) / 2 = e^(-x^2) t Q(t) with
    // t = 1 / (1 + p x) and Q the polynomial of degree 6 that has the least relative error
    // there for x up to 9.7, 6.1e-7 (found by Remez's exchange in 40 digits; p, 0.3725, by
    // trial): below 0 this tail is the result.  Its error is 2^-18 of it in all, and 2^-23
    // z^2 for the exponential's argument.  Past |z| = 14 it is 0, of an infinite z as well.
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const float t = fast_inverse(fmaf(0.26339728f, fabsf(z[j]), 1.0f));
      float q = fmaf(t, -0.06966225845f, 0.2065859024f);
      q = fmaf(t, q, -0.0798374792f);
      q = fmaf(t, q, 0.1506843399f);
      q = fmaf(t, q, 0.07961879453f);
      q = fmaf(t, q, 0.1076840866f);
      q = fmaf(t, q, 0.1049266704f);
      q *= t * fast_exp2(-0.72134752044448170f * (z[j] * z[j]));
      z[j] = fmaf(-fminf(fabsf(z[j]), 14.0f), q, fmaxf(z[j], 0.0f));
    }
  } else if (act == MXFP4_ACT_GELU_TANH) {
    // 0.5 (1 + tanh(v)) = 1 / (1 + e^-2v)
#pragma unroll
    for (int j = 0; j < kCount; ++j)
      z[j] = sigmoid_times(z[j], 1.5957691216057308f * (z[j] + 0.044715f * z[j] * z[j] * z[j]));
  }
}

// 1 / (a b), the global scales' inverse, as alpha * beta for sum * alpha * beta: neither
// overflows or vanishes where the result does not (sum * 1/a * 1/b would: a sum of 2^20
// beside 2^-120 and 2^120).  The mantissas' part and half of the exponent are alpha, the
// other half is beta; off by 2^-24 for the product and 2^-23 for its inverse.  A sum of E2M1 and E4M3 products
// is 0 or 2^-20 to 2^53, so past 2^240 and 2^-240 nothing changes, and a sum of zero
// stays zero beside any of them.
struct Scaling {
  float alpha, beta;
};
// A number's mantissa in [1, 2) with its sign, its exponent (biased by 127) taken from
// `e`; 0, infinity and NaN are their own mantissas.
__device__ __forceinline__ float mantissa_of(float a, int& e) {
  if (fabsf(a) < 0x1p-126f) a *= 0x1p64f, e += 64;
  const int bits = __float_as_int(a), field = (bits >> 23) & 255;
  e -= field;
  return field == 0 || field == 255 ? a : __int_as_float((bits & 0x807FFFFF) | 0x3F800000);
}
__device__ __forceinline__ Scaling scaling_of(float a, float b) {
  int e = 2 * 127;
  const float ma = mantissa_of(a, e), mb = mantissa_of(b, e), m = fast_inverse(ma * mb);
  e = max(-240, min(240, e));
  const int half = e >> 1;
  const auto power = [](int n) { return __int_as_float((n + 127) << 23); };
  return Scaling{m * power(half), power(e - half)};
}

// What a thread's row of the weights adds and scales: z = sum * alpha * beta + bias.
struct RowTerms {
  float alpha, beta, bias, other_bias;  // `other`: of the second half
};
template <bool kNv>
__device__ __forceinline__ Scaling scaling(const GemmParams& p, int e) {
  if (!kNv || p.steps == 0) return Scaling{1.0f, 1.0f};
  return scaling_of(MXFP4_IN_BOUNDS(p, kDbgXGlobals, p.x_globals + e, 4) ? __ldg(p.x_globals + e) : 1.0f,
                    MXFP4_IN_BOUNDS(p.more, kDbgGlobals, p.globals + e, 4) ? __ldg(p.globals + e) : 1.0f);
}
template <bool kGated, bool kF16>
__device__ __forceinline__ RowTerms row_terms(const GemmParams& p, const Tile& t, int n, Scaling g) {
  RowTerms r{g.alpha, g.beta, 0.0f, 0.0f};
  if (p.bias != nullptr && n < p.cols) {
    const uint16_t* at = p.bias + static_cast<int64_t>(t.e) * p.N + n;
    r.bias = MXFP4_IN_BOUNDS(p, kDbgBias, at, 2) ? widen<kF16>(__ldg(at)) : 0.0f;
    if (kGated) {
      at += p.cols;
      r.other_bias = MXFP4_IN_BOUNDS(p, kDbgBias, at, 2) ? widen<kF16>(__ldg(at)) : 0.0f;
    }
  }
  return r;
}

// Activation and gate of z = v (u: the second half's), in place.
template <bool kGated, int kCount>
__device__ __forceinline__ void activate_gate(const GemmParams& p, float (&v)[kCount], float (&u)[kCount]) {
  if constexpr (kGated) {
    if (p.gate_second) activate(u, p.activation);
    else activate(v, p.activation);
#pragma unroll
    for (int j = 0; j < kCount; ++j) v[j] *= u[j];
  } else {
    activate(v, p.activation);
  }
}
// kCount tokens' sums v (u: the second half's) finished in place, but for the residual.
template <bool kGated, int kCount>
__device__ __forceinline__ void finish(const GemmParams& p, const RowTerms& r, float (&v)[kCount],
                                       float (&u)[kCount]) {
#pragma unroll
  for (int j = 0; j < kCount; ++j) v[j] = fmaf(v[j] * r.alpha, r.beta, r.bias);
  if constexpr (kGated) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) u[j] = fmaf(u[j] * r.alpha, r.beta, r.other_bias);
  }
  activate_gate<kGated>(p, v, u);
}

// A thread's kSome tokens of column n from column c of the tile on, two tokens to a
// word.  Where rows lie in whole words, neighbours share the copies: each takes
// both their columns of every other token, and they exchange.  `whole`: none of
// the warp's tokens and columns is outside.
__device__ __forceinline__ uint32_t exchange(uint32_t mine, int odd) {
  return __byte_perm(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 1), odd ? 0x3276 : 0x5410);
}
template <int kSome>
__device__ __forceinline__ bool whole_chunk(const GemmParams& p, const Tile& t, int c) {
  return c + kSome <= t.n && t.r0 + kRows <= p.cols;
}
// The residual added (plain loads: it may be y, of which these are read before they
// are written, by this warp alone).  32 tokens of it were asked into L2 before, a
// row to a lane.
__device__ __forceinline__ void prefetch_residual(const GemmParams& p, const Tile& t, int first, int c) {
  const int lane = threadIdx.x & 31;
  const uint16_t* const at = p.residual + (t.row + c + lane) * p.ldr + first;
  if (c + lane < t.n && first < p.cols && MXFP4_IN_BOUNDS(p, kDbgResidual, at, 2)) prefetch_l2(at);
}
template <bool kF16, int kSome>
__device__ __forceinline__ void add_residual(const GemmParams& p, const Tile& t, int n, int c, float (&v)[kSome]) {
  if (p.paired_residual) {
    const int odd = n & 1;
    const uint16_t* at = p.residual + (t.row + c + odd) * p.ldr + (n & ~1);
    const bool whole = whole_chunk<kSome>(p, t, c);
    uint32_t r[kSome / 2];
#pragma unroll
    for (int j = 0; j < kSome / 2; ++j) {
      r[j] = 0;
      if ((whole || (c + 2 * j + odd < t.n && n < p.cols)) && MXFP4_IN_BOUNDS(p, kDbgResidual, at, 4))
        r[j] = *reinterpret_cast<const uint32_t*>(at);
      at += 2 * p.ldr;
    }
#pragma unroll
    for (int j = 0; j < kSome / 2; ++j) {
      const uint32_t w = exchange(r[j], odd);
      v[2 * j] += widen<kF16>(static_cast<uint16_t>(w));
      v[2 * j + 1] += widen<kF16>(static_cast<uint16_t>(w >> 16));
    }
  } else {
    const uint16_t* at = p.residual + (t.row + c) * p.ldr + n;
#pragma unroll
    for (int q = 0; q < kSome; q += 4) {
      uint16_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = 0;
        if (c + q + j < t.n && n < p.cols && MXFP4_IN_BOUNDS(p, kDbgResidual, at, 2)) r[j] = *at;
        at += p.ldr;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q + j] += widen<kF16>(r[j]);
    }
  }
}
template <bool kF16, int kSome>
__device__ __forceinline__ void store(const GemmParams& p, const Tile& t, int n, int c, const float (&v)[kSome]) {
  if (p.paired && whole_chunk<kSome>(p, t, c)) {
    const int odd = n & 1;
    uint16_t* at = p.y + (t.row + c + odd) * p.ldy + (n & ~1);
#pragma unroll
    for (int j = 0; j < kSome / 2; ++j) {
      const uint32_t word = exchange(narrow2<kF16>(v[2 * j], v[2 * j + 1]), odd);
      if (MXFP4_IN_BOUNDS(p, kDbgY, at, 4)) *reinterpret_cast<uint32_t*>(at) = word;
      at += 2 * p.ldy;
    }
  } else {
    uint16_t* at = p.y + (t.row + c) * p.ldy + n;
#pragma unroll
    for (int j = 0; j < kSome; ++j) {
      if (c + j < t.n && n < p.cols && MXFP4_IN_BOUNDS(p, kDbgY, at, 2))
        *at = static_cast<uint16_t>(narrow2<kF16>(v[j], 0.0f));
      at += p.ldy;
    }
  }
}

// ------------------------------------------------------------------- scales
// A stage's scales as the products need them, where they do not lie so:
// rows `shift` on of the two tiles that the second half spans, moved to the first;
// bytes past the last block of a row, whatever they hold, made zero.
template <bool kNv>
__device__ void mend_scales(uint32_t scales, int tiles, int moved, int shift, int keep) {
  const int lane = threadIdx.x & 31;
  if (shift != 0) {
    const uint32_t lo = scales + moved * Layout<kNv>::kScales, hi = scales + 3 * Layout<kNv>::kScales;
    const int row = (shift + lane) & 31, first = (shift + lane) >> 5;  // first: 0..4
    uint32_t w[Layout<kNv>::kChunks][4];
#pragma unroll
    for (int c = 0; c < Layout<kNv>::kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = first + j;
        w[c][j] = lds32((q < 4 ? lo : hi) + c * 512 + row * 16 + (q & 3) * 4);
      }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < Layout<kNv>::kChunks; ++c)
      sts128(lo + c * 512 + lane * 16, w[c][0], w[c][1], w[c][2], w[c][3]);
    __syncwarp();
  }
  if (keep >= 0) {  // bytes of the row that are scales, in this stage
    const uint32_t mask = (1u << (8 * (keep & 3))) - 1u;  // of the chunk's word that is not full
    for (int i = 0; i < tiles; ++i) {
      const uint32_t at = scales + i * Layout<kNv>::kScales + (keep >> 2) * 512 + lane * 16;
      const uint4 v = lds128(at);
      sts128(at, v.x & mask, v.y & mask, v.z & mask, v.w & mask);
    }
  }
  tc::fence_async();
  __syncwarp();
}

// --------------------------------------------------------------- the kernel
template <bool kNv, bool kGated, bool kF16, bool kAdd>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap w_map,
                const GemmParams p) {
  using L = Layout<kNv>;
  constexpr int kTokens = kGated ? 128 : 256;
  constexpr int kWeightSlabs = kGated ? 2 : 1;
  extern __shared__ uint8_t smem[];
  __shared__ Barriers bars;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t ring = (tc::shared_address(smem) + 1023u) & ~1023u;
  const auto bar = [](const uint64_t& b) { return tc::shared_address(&b); };
  uint32_t ranks;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const uint32_t rank = ranks > 1 ? cluster_rank() : 0;
  const int first_tile = ranks > 1 ? static_cast<int>(blockIdx.x / ranks) : static_cast<int>(blockIdx.x);
  const int tile_step = ranks > 1 ? INT32_MAX / 2 : static_cast<int>(gridDim.x);  // clusters: one tile
  const int k_begin = static_cast<int>(static_cast<int64_t>(p.stages) * rank / ranks);
  const int k_end = static_cast<int>(static_cast<int64_t>(p.stages) * (rank + 1) / ranks);

  // the second half's rows begin at row `shift` of a tile of the scales
  const int shift = kGated ? p.cols & (kRows - 1) : 0;
  // a product's 64 elements of K go past the last scale
  const bool tail = (p.blocks & (kNv ? 3 : 1)) != 0;
  const bool mended = shift != 0 || tail;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      tc::barrier_init(bar(bars.full[s]), 1);
      tc::barrier_init(bar(bars.mended[s]), 1);
      tc::barrier_init(bar(bars.empty[s]), 1);
    }
    tc::barrier_init(bar(bars.sums_full), 1);
    tc::barrier_init(bar(bars.sums_empty), kEpilogueWarps);
    for (int i = 0; i < kJobs; ++i) {
      tc::barrier_init(bar(bars.job_full[i]), 1);
      tc::barrier_init(bar(bars.job_empty[i]), 2 + mended + kEpilogueWarps);
    }
    tc::barrier_init(bar(bars.drained), 1);
    tc::barrier_init_fence();
    bars.gave_up = 0;
    bars.job[0].t.n = -1;
    if (p.stages > 0 && p.rows > 0 && p.E > 0 && p.N > 0) tc::prefetch_map(&x_map), tc::prefetch_map(&w_map);
  }
  if (warp == 1) tc::allocate(tc::shared_address(&bars.columns), kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t gave_up = tc::shared_address(&bars.gave_up);
  pdl_wait();
  pdl_release();

  bool work = true;
  if (p.offsets != nullptr) {
    int bad = threadIdx.x == 0 && offset_at(p, 0) != 0;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
      const int from = offset_at(p, e), to = offset_at(p, e + 1);
      bad |= from < 0 || from > to || to > p.rows;
    }
    work = __syncthreads_or(bad) == 0;
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.status != nullptr && MXFP4_IN_BOUNDS(p, kDbgStatus, p.status, 4))
      *p.status = work ? MXFP4_OK : MXFP4_EOFFSETS;
  }
  Tile t{};
  uint32_t copied = 0;  // stages, by this thread
  if (!work) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (tc::elected()) {
      const int64_t row_bytes = static_cast<int64_t>(p.nKT) * 512, begin = static_cast<int64_t>(k_begin) * L::kScales;
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (uint32_t j = 0; ok; ++j) {
        ok = tc::barrier_wait(bar(bars.job_full[j % kJobs]), j / kJobs & 1u, gave_up);
        if (!ok) break;
        const Job job = bars.job[j % kJobs];
        tc::barrier_arrive(bar(bars.job_empty[j % kJobs]));
        if (job.t.n < 0 || stalled(kStallCopies)) break;
        const int boxes = (job.t.n + p.box_rows - 1) / p.box_rows;
        const uint32_t box_bytes = p.box_rows * kStageBytes;
        // the tiles' scales: of the weights (both halves'), of the tokens, and of the
        // tile behind the second half's first where it does not begin at a tile and
        // is not the last
        const uint8_t* const ws = p.scales + begin;
        const uint8_t* const xs = p.x_scales + job.x_scales + begin;
        const uint8_t* src[4] = {ws + job.scales, kGated ? ws + job.upper : xs, kGated ? xs : xs + row_bytes,
                                 ws + job.upper + row_bytes};
        const bool third = kGated || job.t.n > kRows;
        const bool fourth = kGated && shift != 0 && (p.cols + job.t.r0) / kRows * kRows + kRows < p.N;
        const uint32_t code_bytes = kWeightSlabs * kSlab + boxes * box_bytes;
        const uint32_t scale_tiles = 2 + third + fourth;
        for (int k = k_begin; k < k_end; ++k, ++copied) {
          if (copied >= p.ring_stages && !(ok = tc::barrier_wait(bar(bars.empty[stage]), phase ^ 1u, gave_up))) break;
          const uint32_t at = ring + stage * p.stage_bytes, sc = at + p.scales_at, full = bar(bars.full[stage]);
          const uint32_t bytes = min(L::kChunks, p.nKT - k * L::kChunks) * 512;
          bool whole = true;  // of the buffers: false only in the bounds-checking build
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (s < 2 || (s == 2 && third) || (s == 3 && fourth))
              whole &= MXFP4_IN_BOUNDS(p, (kGated ? s == 2 : s > 0) ? kDbgXScales : kDbgScales, src[s], bytes);
          tc::barrier_expect(full, code_bytes + (whole ? scale_tiles * bytes : 0));
          const int x = k * kStageBytes;
          tc::copy_box(at, &w_map, x, job.w_row, full);
          if constexpr (kGated) tc::copy_box(at + kSlab, &w_map, x, job.w_row + p.cols, full);
          for (int b = 0; b < boxes; ++b)
            tc::copy_box(at + kWeightSlabs * kSlab + b * box_bytes, &x_map, x, job.t.row + b * p.box_rows, full);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if ((s < 2 || (s == 2 && third) || (s == 3 && fourth)) && whole)
              tc::copy_bytes(sc + s * L::kScales, src[s], bytes, full);
            src[s] += L::kScales;
          }
          if (++stage == p.ring_stages) stage = 0, phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    // One thread issues them, and its instructions are their pace.
    if (tc::elected()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (uint32_t j = 0; ok; ++j) {
        ok = tc::barrier_wait(bar(bars.job_full[j % kJobs]), j / kJobs & 1u, gave_up);
        if (!ok) break;
        const int n = bars.job[j % kJobs].t.n;
        tc::barrier_arrive(bar(bars.job_empty[j % kJobs]));
        if (n < 0 || stalled(kStallProducts)) break;
        if (k_begin == k_end) continue;
        if (j > 0) ok = tc::barrier_wait(bar(bars.sums_empty), (j - 1) & 1u, gave_up);  // the tile's before
        tc::fence_after();
        const uint32_t inst = tc::instruction((n + 15) / 16 * 16, kNv), inst_odd = tc::with_scale_byte(inst, 2);
        const bool wide = n > kRows;
        for (int k = k_begin; ok && k < k_end; ++k) {
          ok = tc::barrier_wait(mended ? bar(bars.mended[stage]) : bar(bars.full[stage]), phase, gave_up);
          if (!ok) break;
          tc::fence_after();
          const uint32_t at = ring + stage * p.stage_bytes;
          const uint32_t a = tc::operand_low(at), b = a + kWeightSlabs * kSlab / 16;
          const uint32_t s0 = tc::scales_low(at + p.scales_at);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c) {  // (past the last chunk: what no product uses)
            constexpr uint32_t kTile = L::kScales / 16;  // a tile's scales
            const auto from = [&](int tile) { return tc::descriptor(s0 + tile * kTile + c * 32, tc::kScalesHigh); };
            tc::copy_scales(kScalesA + c * 4, from(0));
            if constexpr (kGated) {
              tc::copy_scales(kScalesA + 16 + c * 4, from(1));
              tc::copy_scales(kScalesB + c * 4, from(2));
            } else {
              tc::copy_scales(kScalesB + c * 8, from(1));
              if (wide) tc::copy_scales(kScalesB + c * 8 + 4, from(2));
            }
          }
          const int steps = p.steps - k * kSteps;
          constexpr int kStride = kGated ? 4 : 8;  // the tokens' columns of a chunk
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            if (s >= steps) continue;
            const int c = kNv ? s : s >> 1;
            const uint32_t in = kNv || (s & 1) == 0 ? inst : inst_odd;
            const bool add = s > 0 || k > k_begin;
            const uint64_t bd = tc::descriptor(b + 2 * s, tc::kOperandHigh);
            tc::multiply<kNv>(0, tc::descriptor(a + 2 * s, tc::kOperandHigh), bd, in, kScalesA + c * 4,
                              kScalesB + c * kStride, add);
            if constexpr (kGated)
              tc::multiply<kNv>(kSecond, tc::descriptor(a + kSlab / 16 + 2 * s, tc::kOperandHigh), bd, in,
                                kScalesA + 16 + c * 4, kScalesB + c * kStride, add);
          }
          tc::arrive_when_done(bar(bars.empty[stage]));
          if (++stage == p.ring_stages) stage = 0, phase ^= 1u;
        }
        if (ok) tc::arrive_when_done(bar(bars.sums_full));
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------- scales that do not lie as they should
    uint32_t count = 0;
    bool ok = mended;
    for (uint32_t j = 0; ok; ++j) {
      ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait(bar(bars.job_full[j % kJobs]), j / kJobs & 1u, gave_up));
      if (!ok) break;
      const int n = bars.job[j % kJobs].t.n;
      __syncwarp();
      if (lane == 0) tc::barrier_arrive(bar(bars.job_empty[j % kJobs]));
      if (n < 0) break;
      for (int k = k_begin; ok && k < k_end; ++k, ++count) {
        const uint32_t stage = count % p.ring_stages;
        ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait(bar(bars.full[stage]), count / p.ring_stages & 1u, gave_up));
        if (!ok) break;
        const int keep = k == p.stages - 1 && tail ? p.blocks - k * L::kChunks * 4 : -1;
        if (shift != 0 || keep >= 0) mend_scales<kNv>(ring + stage * p.stage_bytes + p.scales_at, 3, 1, shift, keep);
        if (lane == 0) tc::barrier_arrive(bar(bars.mended[stage]));
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------- the tiles
    Walk walk;
    const int64_t row_bytes = static_cast<int64_t>(p.nKT) * 512;
    bool ok = true, more = true;
    uint32_t j = 0;
    for (int i = first_tile; ok && more; i += tile_step, ++j) {
      more = walk.find(p, i, t);
      if (!more) t.n = -1;
      if (stalled(kStallTiles)) break;
      if (lane == 0) {
        if (j >= kJobs) ok = tc::barrier_wait(bar(bars.job_empty[j % kJobs]), (j / kJobs - 1) & 1u, gave_up);
        if (ok) {
          const int64_t scales = t.e * p.expert_scales;
          bars.job[j % kJobs] = Job{t, t.e * p.N + t.r0, scales + t.r0 / kRows * row_bytes,
                                    scales + (p.cols + t.r0) / kRows * row_bytes, t.padded / kRows * row_bytes};
          tc::barrier_arrive(bar(bars.job_full[j % kJobs]));
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
  } else if (warp >= kFirstEpilogue) {
    // ---------------------------------------------------------- epilogue
    // A warp has a quarter of the rows and one or two chunks of 32 tokens, whose
    // sums it takes at once: tensor memory is the next tile's before they are
    // finished and stored.
    constexpr int kChunks = kTokens / 128;
    // tokens finished at a time: as many as the registers hold (16 for 8: a tile's
    // epilogue 3.0 -> 2.2 us)
    constexpr int kSome = (kGated ? 8 : 16) / (kAdd ? kNv && !kGated ? 4 : 2 : 1);
    const int group = (warp - kFirstEpilogue) >> 2, quarter = warp & 3;
    const uint32_t from = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    for (uint32_t j = 0; ok; ++j) {
      ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait(bar(bars.job_full[j % kJobs]), j / kJobs & 1u, gave_up));
      if (!ok) break;
      t = bars.job[j % kJobs].t;
      __syncwarp();
      if (lane == 0) tc::barrier_arrive(bar(bars.job_empty[j % kJobs]));
      if (t.n < 0) break;
      const int n = t.r0 + quarter * 32 + lane;
      const RowTerms terms = row_terms<kGated, kF16>(p, t, n, scaling<kNv>(p, t.e));
      if (kAdd && ranks == 1) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) prefetch_residual(p, t, t.r0 + quarter * 32, group * 32 + 128 * c);
      }
      // gated: of the first half, then of the second
      float sums[64];
      if (p.stages > 0) {
        ok = __all_sync(0xFFFFFFFFu, tc::barrier_wait(bar(bars.sums_full), j & 1u, gave_up));
        if (!ok) break;
        tc::fence_after();
        tc::load_sums(from + group * 32, from + kSecond + group * 32, sums);
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) sums[j] = 0.0f;
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::barrier_arrive(bar(bars.sums_empty));
#pragma unroll
      for (int some = 0; some < kChunks * 32; some += kSome) {
        const int column = group * 32 + (some & 31) + (some & 32) * 4;
        if (column >= t.n) break;
        auto& v = *reinterpret_cast<float(*)[kSome]>(sums + some);
        auto& u = *reinterpret_cast<float(*)[kSome]>(sums + (kGated ? 32 + some : 0));
        if (ranks > 1) {
          // this CTA's part of the sums to its shared memory, [token][row]: the
          // ring is free, all its products are done
#pragma unroll
          for (int j = 0; j < kSome; ++j) {
            const uint32_t at = ring + ((column + j) * kRows + quarter * 32 + lane) * 4;
            sts32(at, __float_as_uint(v[j]));
            if constexpr (kGated) sts32(at + kTokens * kRows * 4, __float_as_uint(u[j]));
          }
        } else {
          finish<kGated>(p, terms, v, u);
          if constexpr (kAdd) add_residual<kF16>(p, t, n, column, v);
          store<kF16>(p, t, n, column, v);
        }
      }
    }
  }
  if (ranks > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= kFirstEpilogue && bars.job[0].t.n > 0) {  // a cluster has one tile or none
      t = bars.job[0].t;
      // Each rank finishes every ranks-th token, a warp of it every 16th of those, a
      // thread four rows: the parts of all ranks in flight at once, added in order.
      constexpr int kSome = 4, kMaxRanks = 8;
      const int n = t.r0 + lane * kSome;
      RowTerms terms[kSome];
      const Scaling g = scaling<kNv>(p, t.e);
#pragma unroll
      for (int j = 0; j < kSome; ++j) terms[j] = row_terms<kGated, kF16>(p, t, n + j, g);
      // (asked for ahead of the parts, looked at behind them)
      const bool lost = lane < static_cast<int>(ranks) && tc::raised_there(gave_up, lane);
      for (int c = rank + ranks * (warp - kFirstEpilogue); c < t.n; c += ranks * kEpilogueWarps) {
        float4 a[kMaxRanks], b[kMaxRanks];
#pragma unroll
        for (uint32_t r = 0; r < kMaxRanks; ++r)
          if (r < ranks) {
            const uint32_t at = cluster_address(ring, r) + (c * kRows + lane * kSome) * 4;
            a[r] = ld_cluster_f4(at);
            if constexpr (kGated) b[r] = ld_cluster_f4(at + kTokens * kRows * 4);
          }
        float v[kSome] = {}, u[kSome] = {};
        if (__any_sync(0xFFFFFFFFu, lost)) {  // a rank has not its part
#pragma unroll
          for (int j = 0; j < kSome; ++j) v[j] = u[j] = NAN;
        }
#pragma unroll
        for (uint32_t r = 0; r < kMaxRanks; ++r)
          if (r < ranks) {
            v[0] += a[r].x, v[1] += a[r].y, v[2] += a[r].z, v[3] += a[r].w;
            if constexpr (kGated) u[0] += b[r].x, u[1] += b[r].y, u[2] += b[r].z, u[3] += b[r].w;
          }
#pragma unroll
        for (int j = 0; j < kSome; ++j) {
          v[j] = fmaf(v[j] * terms[j].alpha, terms[j].beta, terms[j].bias);
          if constexpr (kGated) u[j] = fmaf(u[j] * terms[j].alpha, terms[j].beta, terms[j].other_bias);
        }
        activate_gate<kGated>(p, v, u);
        if constexpr (kAdd) {
          const uint16_t* const at = p.residual + (t.row + c) * p.ldr + n;
#pragma unroll
          for (int j = 0; j < kSome; ++j)
            if (n + j < p.cols && MXFP4_IN_BOUNDS(p, kDbgResidual, at + j, 2)) v[j] += widen<kF16>(at[j]);
        }
        uint16_t* const at = p.y + (t.row + c) * p.ldy + n;
#pragma unroll
        for (int j = 0; j < kSome; j += 2) {
          const uint32_t word = narrow2<kF16>(v[j], v[j + 1]);
          if (p.paired) {
            if (n + j < p.cols && MXFP4_IN_BOUNDS(p, kDbgY, at + j, 4)) *reinterpret_cast<uint32_t*>(at + j) = word;
          } else {
            if (n + j < p.cols && MXFP4_IN_BOUNDS(p, kDbgY, at + j, 2)) at[j] = static_cast<uint16_t>(word);
            if (n + j + 1 < p.cols && MXFP4_IN_BOUNDS(p, kDbgY, at + j + 1, 2)) at[j + 1] = static_cast<uint16_t>(word >> 16);
          }
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (tc::raised(gave_up)) {
    // A wait ran out.  What was issued is done before the CTA may end, all of its tiles
    // are NaN, and the status word says so.
    if (warp == 0)
      for (uint32_t n = copied > p.ring_stages ? copied - p.ring_stages : 0; n < copied; ++n)
        tc::barrier_wait_alone(bar(bars.full[n % p.ring_stages]), n / p.ring_stages & 1u);
    if (warp == 1 && tc::elected()) {
      tc::arrive_when_done(bar(bars.drained));
      tc::barrier_wait_alone(bar(bars.drained), 0);
    }
    Walk walk;
    for (int i = first_tile; walk.find(p, i, t); i += tile_step)
      for (int r = warp; r < t.n; r += kThreads / 32)
        for (int n = t.r0 + lane; n < min(t.r0 + kRows, p.cols); n += 32) {
          uint16_t* const at = p.y + (t.row + r) * p.ldy + n;
          if (MXFP4_IN_BOUNDS(p, kDbgY, at, 2)) *at = 0x7FFF;
        }
    if (threadIdx.x == 0 && p.status != nullptr && MXFP4_IN_BOUNDS(p, kDbgStatus, p.status, 4))
      *p.status = MXFP4_ECUDA;
    __syncthreads();
  }
  if (warp == 1) tc::release(bars.columns, kColumns);
}

// ------------------------------------------------------------------- launch
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled found = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  return found;
}

// Rows of K/2 bytes of codes, in boxes of 128 bytes by `box` rows; zeros outside.
cudaError_t map_codes(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t boxes[2] = {kStageBytes, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// How many clusters of `ranks` such CTAs (one to an SM) the current device runs at
// once; asked of the runtime once per device and size.
int clusters_at_once(const void* kernel, int bytes, int ranks) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  std::atomic<int>& place = known[dev][ranks == 2 ? 1 : ranks == 4 ? 2 : 3];
  int n = place.load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(ranks), 1u, 1u};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  place.store(n + 1, std::memory_order_relaxed);
  return n;
}

template <bool kNv, bool kGated, bool kF16, bool kAdd>
cudaError_t launch_typed(const CUtensorMap& x_map, const CUtensorMap& w_map, const GemmParams& p, int64_t tiles,
                         cudaStream_t stream) {
  constexpr int kBytes = kRingBytes + 1024;  // the ring begins at a multiple of 1024
  static std::atomic<uint64_t> ready{0};
  if (const cudaError_t e = allow_smem(gemm_kernel<kNv, kGated, kF16, kAdd>, kBytes, ready); e != cudaSuccess) return e;
  // Clusters that share a tile's K: two stages to a CTA or more (2048 x 768 by 1 token:
  // 3.7 us, in clusters of 2 4.6), and only as many CTAs as run at once (16 clusters of 8
  // do not, on these 152 SMs: 2048 x 7168 by 16 tokens 10.8 us, in clusters of 4 5.9).
  const int64_t sms = sm_count();
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= sms && ranks * 4 <= p.stages &&
         tiles <= clusters_at_once(reinterpret_cast<const void*>(gemm_kernel<kNv, kGated, kF16, kAdd>), kBytes, ranks * 2))
    ranks *= 2;
  const int64_t grid = ranks > 1 ? tiles * ranks : tiles < sms ? tiles : sms;
  return launch_pdl_cluster(gemm_kernel<kNv, kGated, kF16, kAdd>, dim3(static_cast<unsigned>(grid)), kThreads, kBytes, stream,
                            ranks > 1 ? ranks : 0, x_map, w_map, p);
}

}  // namespace

cudaError_t launch_gemm(const GemmArgs& a, cudaStream_t stream) {
  GemmParams p{};
  const bool gated = a.gate != MXFP4_GATE_NONE;
  p.x_scales = a.x_scales;
  p.scales = a.scales;
  p.x_globals = a.x_globals;
  p.globals = a.globals;
  p.offsets = a.offsets;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.y = static_cast<uint16_t*>(a.y);
  p.status = a.status;
  p.ldr = a.ldr;
  p.ldy = a.ldy;
  p.rows = static_cast<int32_t>(a.rows);
  p.N = static_cast<int32_t>(a.N);
  p.cols = gated ? p.N / 2 : p.N;
  p.E = a.E;
  p.blocks = static_cast<int32_t>(a.K / (a.nvfp4 ? 16 : 32));
  p.nKT = (p.blocks + 3) / 4;
  p.steps = static_cast<int32_t>((a.K + 63) / 64);
  p.stages = (p.steps + kSteps - 1) / kSteps;
  p.row_tiles = (p.cols + kRows - 1) / kRows;
  p.expert_scales = (a.N + 127) / 128 * p.nKT * static_cast<int64_t>(kChunkBytes);
  p.activation = a.activation;
  p.gate_second = a.gate == MXFP4_GATE_SECOND;
  p.paired_residual = p.cols % 2 == 0 && a.ldr % 2 == 0 && reinterpret_cast<uintptr_t>(a.residual) % 4 == 0;
  p.paired = p.cols % 2 == 0 && a.ldy % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % 4 == 0;
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.dbg, kDbgXScales, a.x_scales,
              (a.rows + 127 * static_cast<int64_t>(a.E)) / 128 * p.nKT * kChunkBytes);
  debug_range(p.dbg, kDbgScales, a.scales, a.E * p.expert_scales);
  debug_range(p.dbg, kDbgOffsets, a.offsets, a.offsets ? (static_cast<int64_t>(a.E) + 1) * 4 : 0);
  debug_range(p.dbg, kDbgBias, a.bias, a.bias ? a.E * a.N * 2 : 0);
  debug_range(p.dbg, kDbgResidual, a.residual, a.residual ? ((a.rows - 1) * a.ldr + p.cols) * 2 : 0);
  debug_range(p.dbg, kDbgY, a.y, a.rows > 0 ? ((a.rows - 1) * a.ldy + p.cols) * 2 : 0);
  debug_range(p.dbg, kDbgStatus, a.status, a.status ? 4 : 0);
  debug_range(p.dbg, kDbgXGlobals, a.x_globals, a.nvfp4 ? a.E * 4 : 0);
  debug_range(p.more.dbg, kDbgGlobals, a.globals, a.nvfp4 ? a.E * 4 : 0);
#endif
  // Rows to a copy of x: many in one where experts have many, few where whole
  // boxes would be other experts' rows.  Tiles of 128 tokens where
  // the SMs hold them all: a tile is done sooner, and its stages are smaller (512 tokens
  // by 2881 x 2880 12.9 -> 9.5 us; 600 by 4096 x 4096, 160 of them, 13.3 -> 15.3).  Not
  // for experts with fewer tokens on average: some have more, and twice the tiles (2000
  // tokens' 8 routes to 128 experts, down products 38 -> 42).
  const int64_t average = a.offsets ? a.rows / (a.E > 0 ? a.E : 1) : a.rows;
  p.box_rows = average > 64 ? 128 : 32;
  const bool few = !a.offsets && (a.rows + 127) / 128 * p.row_tiles <= sm_count();
  p.tile_tokens = gated || few ? 128 : 256;
  const int64_t slab_rows = std::min<int64_t>(p.tile_tokens, (a.rows + p.box_rows - 1) / p.box_rows * p.box_rows);
  p.scales_at = static_cast<uint32_t>((gated ? 2 : 1) * kSlab + slab_rows * kStageBytes);
  p.stage_bytes = p.scales_at + (gated ? 4 : 3) * (a.nvfp4 ? Layout<true>::kScales : Layout<false>::kScales);
  p.ring_stages = std::min<uint32_t>(kMaxStages, kRingBytes / p.stage_bytes);
  CUtensorMap x_map{}, w_map{};
  if (a.K > 0 && a.rows > 0 && a.N > 0 && a.E > 0) {
    if (const cudaError_t e = map_codes(&x_map, a.x_codes, a.rows, a.K, p.box_rows); e != cudaSuccess) return e;
    if (const cudaError_t e = map_codes(&w_map, a.codes, a.E * a.N, a.K, kRows); e != cudaSuccess) return e;
  }
  // at most this many tiles: every expert with rows may have one that is not full
  const int64_t token_tiles = a.offsets ? a.rows / p.tile_tokens + (a.rows < a.E ? a.rows : a.E)
                                        : (a.rows + p.tile_tokens - 1) / p.tile_tokens;
  int64_t tiles = token_tiles * p.row_tiles;
  if (tiles < 1) tiles = 1;  // the status word alone
  using std::false_type, std::true_type;
  const auto launch = [&](auto nv, auto gate, auto f16, auto add) {
    return launch_typed<decltype(nv)::value, decltype(gate)::value, decltype(f16)::value, decltype(add)::value>(
        x_map, w_map, p, tiles, stream);
  };
  const auto with_add = [&](auto nv, auto gate, auto f16) {
    return a.residual ? launch(nv, gate, f16, true_type{}) : launch(nv, gate, f16, false_type{});
  };
  const auto with_type = [&](auto nv, auto gate) {
    return a.f16 ? with_add(nv, gate, true_type{}) : with_add(nv, gate, false_type{});
  };
  if (a.nvfp4) return gated ? with_type(true_type{}, true_type{}) : with_type(true_type{}, false_type{});
  return gated ? with_type(false_type{}, true_type{}) : with_type(false_type{}, false_type{});
}

#ifdef MXFP4_DEBUG_BOUNDS
bool debug_stall_gemm(int role) { return cudaMemcpyToSymbol(g_debug_stall, &role, sizeof role) == cudaSuccess; }

unsigned int debug_violations_gemm() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

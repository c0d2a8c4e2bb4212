// matvec.cu — products of a few tokens with 4-bit weights (MXFP4 or NVFP4),
// dense and per expert segment, for sm_103a.
//
//   y[r, n] = sum_k x[r, k] * W[n, k]
//   MXFP4: W = e2m1(code) * 2^(s-127), one scale byte per 32 elements of K
//   NVFP4: W = e2m1(code) * e4m3(s) / g, one scale byte per 16 elements
// Sums are float32; the result is rounded once to the output's type.
//
// What bounds it: every weight byte is read once and used for T tokens, so
// for few tokens HBM does.  At 6.8 TB/s an SM has to decode and multiply
// about 45 weights a clock, which leaves no room for scalar multiply-adds on
// each token; the tensor cores' m16n8k16 form takes 16 weight rows by 8
// tokens, and a weight costs one conversion (two codes to two halves) for any
// number of tokens up to 8.
//
// A warp owns 16 rows of W and a range of K, and streams its codes through
// its own ring of shared-memory stages (16-byte asynchronous copies, 256
// elements of K by 16 rows each), so warps never wait on one another inside a
// product.  The 16 rows are {4j..4j+3} + {0, 32, 64, 96} of a 128-row tile:
// their scale bytes are 64 consecutive bytes of the tiled layout.
//
// x is staged once per CTA as halves: the order of k inside a 32-element
// block is free as long as both operands agree, so a lane's 4-byte word of
// codes (8 elements) meets the 16 bytes of x at the same place.  BF16 has
// more exponents than a half: each 32-element block of a token is scaled by
// the power of two that puts its largest element in [2^15, 2^16) (11 bits hold
// BF16's 8 exactly down to 2^-32 of that; below, to 2^-40), and the power is
// multiplied back in float32.  Where a token's whole x lies within 2^32, one
// power serves all of it and is multiplied back at the end.
// The MXFP4 scale is a power of two of any size, so it is applied in float32
// to the 32-element partial sums; the E4M3 scale times an E2M1 value has at
// most 6 bits and fits a half, so NVFP4 weights are scaled before the product.
//
// Measured (device time, weights not in L2, call after call): 64000 x 7168 MXFP4 by
// 1 BF16 token 45 us, 5.4 TB/s of 244 MB (48 alone, from flushed caches); the copies
// alone take most of that, the products alone 35 us.  By 16 tokens 70 us (FP16 59):
// 60 % of the cycles issue, with x in panels.  7168 x 7168 by 1 token 11.3 us, the 128 experts'
// 1536 x 2048 NVFP4 by 64 tokens of 8 experts each 46.9 us (4.6 TB/s), 2048 x 768
// by 1 token 5.2 us.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fragments.cuh"
#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"

namespace mxfp4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                      // weight rows of a warp's tile
constexpr int kChunk = 256;                    // elements of K per stage
constexpr int kBlocks = kChunk / 32;
// A row's 128 bytes of codes in a stage, 144 bytes apart: the eight rows that a
// fragment's words come from then lie in different banks.
constexpr int kRowPitch = 144;
constexpr int kStageCodes = kTile * kRowPitch;
constexpr int kStages = 2;     // of a warp's ring (three: no faster, and less room for x)
constexpr int kMaxUnits = 16;  // of a phase
constexpr int kMaxRows = 64;   // of x, of a phase

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
  int64_t expert_codes;   // bytes of one expert's codes
  int64_t expert_scales;  // bytes of one expert's tiled scales
  int32_t rows;
  int32_t N;
  int32_t K;
  int32_t E;
  int32_t nKT;        // 4-column scale chunks of a row
  int32_t tiles;      // 16-row tiles of N (8 per 128 rows)
  int32_t chunks;     // 256-element chunks of K
  int32_t panel;      // chunks of x staged at a time
  int32_t panels;
  int32_t batch;      // tiles of a phase at most, with several panels
  int32_t x_rows;     // token rows that x's shared memory holds
  int32_t x_pitch;    // bytes between them
  int32_t few;        // a stage to a warp at most: x is scaled by block at once
  int32_t y_f32;
  int32_t half_rows;  // rows of codes start at 8-byte (not 16-byte) boundaries
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgX = 0, kDbgCodes, kDbgScales, kDbgGlobal, kDbgY, kDbgIndex, kDbgOffsets, kDbgStatus };

__device__ __forceinline__ int32_t offset_at(const MatvecParams& p, int e) {
  const int32_t* at = p.offsets + e;
  return MXFP4_IN_BOUNDS(p, kDbgOffsets, at, 4) ? __ldg(at) : 0;
}
__device__ __forceinline__ int32_t index_at(const MatvecParams& p, int64_t r) {
  const int32_t* at = p.row_index + r;
  return MXFP4_IN_BOUNDS(p, kDbgIndex, at, 4) ? __ldg(at) : -1;
}

// The rows of one unit of work: up to 8*NT consecutive rows of one segment;
// `x`: the first of its rows of x's shared memory.
struct UnitRows {
  int e, row0, n, x;
};

struct Shared {
  int32_t prefix[kThreads];  // units up to and with each thread's experts
  int32_t warp_sum[kWarps];
  UnitRows unit[kMaxUnits];  // of the phase
  int32_t n_units, n_rows;
  int64_t x_row[kMaxRows];   // x's row of each staged row (-1: none)
  int32_t x_unit[kMaxRows];  // and its unit (-1: padding)
  uint32_t x_max[kMaxRows];  // BF16: largest magnitude of a row, and smallest but zero, less one
  uint32_t x_min[kMaxRows];
  uint32_t unit_max[kMaxUnits];  // MXFP4: largest exponent of a unit's rows
  float x_scale[kMaxRows];   // what undoes a row's scaling (MXFP4: beyond the unit's)
  float unit_scale[kMaxUnits];
  float unit_inverse[kMaxUnits];  // NVFP4: 1 / global scale
  int32_t far;               // BF16: some row needs a power of two for each block
};

// Expert and rows of unit u, from the prefix sums (same result in all lanes).
template <int NT>
__device__ __forceinline__ UnitRows find_unit(const MatvecParams& p, const Shared& s, int u) {
  constexpr int R = 8 * NT;
  UnitRows r;
  r.x = 0;
  if (p.offsets == nullptr) {
    r.e = 0;
    r.row0 = u * R;
    r.n = min(R, p.rows - r.row0);
    return r;
  }
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s.prefix[mid] > u) hi = mid; else lo = mid + 1;
  }
  int base = lo > 0 ? s.prefix[lo - 1] : 0;
  const int per = (p.E + kThreads - 1) / kThreads;
  int e = lo * per;
  for (;; ++e) {
    const int a = offset_at(p, e), n = offset_at(p, e + 1) - a;
    const int c = (n + R - 1) / R;
    if (base + c > u || e + 1 >= p.E) {
      r.e = e;
      r.row0 = a + (u - base) * R;
      r.n = min(R, a + n - r.row0);
      return r;
    }
    base += c;
  }
}

// The warp w whose share [total * w / kWarps, total * (w + 1) / kWarps) holds f.
__device__ __forceinline__ int share_of(int f, int total) { return ((f + 1) * kWarps - 1) / total; }

// Where a warp's copies stand in its share of a phase, and what its lanes copy next.
struct Cursor {
  int panel, f;              // the panel of x; where the run after this one starts
  int chunk, left;           // the next chunk, and the chunks left of this run (one tile's)
  int quarters;              // of the tile's four 32-row quarters, those in which this lane's row is in N
  bool whole;                // all lanes' rows are in N, and start at 16-byte boundaries
  const uint8_t* row;        // this lane's piece of its row of the first quarter, of the next chunk
  const uint8_t* scale;
};

template <bool kNv, bool kF16, int NT>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(const MatvecParams p) {
  constexpr int R = 8 * NT;
  constexpr int kScaleBytes = kNv ? 256 : 128;
  constexpr int kChunkKt = kChunk / (kNv ? 64 : 128);  // 4-column scale chunks of a stage
  constexpr int kStage = kStageCodes + kScaleBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // shared memory: rings | x halves | x block scales | parts of sums
  constexpr int ring_bytes = kStages * kStage;
  const uint32_t ring = smem_u32(smem) + warp * ring_bytes;
  uint8_t* const x_s = smem + kWarps * ring_bytes;
  static_assert(sizeof(Shared) <= 5 * 1024, "kMaxSmem leaves this much");
  float* const xs_s = reinterpret_cast<float*>(x_s + p.x_rows * p.x_pitch);
  float4* const part_s = reinterpret_cast<float4*>(xs_s + (kF16 ? 0 : p.panel * kBlocks * p.x_rows));

  pdl_wait();
  pdl_release();

  // units of work: token chunks of the experts that have rows
  int units;
  if (p.offsets == nullptr) {
    units = (p.rows + R - 1) / R;
  } else {
    const int per = (p.E + kThreads - 1) / kThreads;
    int sum = 0, bad = 0;
    for (int i = 0; i < per; ++i) {
      const int e = threadIdx.x * per + i;
      if (e >= p.E) break;
      const int a = offset_at(p, e), b = offset_at(p, e + 1);
      if (a < 0 || b < a || b > p.rows || (e == 0 && a != 0)) bad = 1;
      else sum += (b - a + R - 1) / R;
    }
    if (p.E == 0 && threadIdx.x == 0 && offset_at(p, 0) != 0) bad = 1;
    bad = __syncthreads_or(bad);
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    int before = 0;
    units = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      units += sh.warp_sum[w];
    }
    sh.prefix[threadIdx.x] = before + scan;
    if (blockIdx.x == 0 && p.status != nullptr) {
      int wrong = 0;
      if (!bad && p.row_index != nullptr) {
        const int used = p.E > 0 ? offset_at(p, p.E) : 0;
        for (int r = threadIdx.x; r < used; r += kThreads) {
          const int32_t i = index_at(p, r);
          if (i < 0 || i >= p.src_rows) wrong = 1;
        }
      }
      wrong = __syncthreads_or(wrong);
      if (threadIdx.x == 0 && MXFP4_IN_BOUNDS(p, kDbgStatus, p.status, 4)) *p.status = bad ? -6 : wrong ? -7 : 0;
    }
    if (bad) return;
    __syncthreads();
  }

  // This CTA's tiles, consecutive over the units, in phases: as many units as x
  // has room for (one, with x in panels).  A phase's tiles times chunks are one
  // sequence of stages of which each warp has an even share, whatever the
  // sizes; a tile whose stages are shared is summed over its warps at the end.
  const int64_t all = static_cast<int64_t>(units) * p.tiles;
  int at = static_cast<int>(all * blockIdx.x / gridDim.x);
  const int last = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x);
  const int n = p.panel;  // chunks of a tile in a panel
  const int tail = p.K % kChunk != 0 ? p.chunks - 1 : -1;  // the chunk that ends before its stage

  while (at < last) {
    // ---- the phase's units, and their rows of x
    const int u0 = at / p.tiles, tile0 = at - u0 * p.tiles;
    __syncthreads();  // the phase before is done with the tables and the sums
    if (warp == 0) {
      UnitRows u{0, 0, 0, 0};
      const int most = p.panels > 1 ? 1 : kMaxUnits;
      const bool there = lane < most && static_cast<int64_t>(u0 + lane) * p.tiles < last;
      if (there) u = find_unit<NT>(p, sh, u0 + lane);
      int x = (u.n + 1) & ~1, sum = x;  // an even number of rows: pairs of factors stay together
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      u.x = sum - x;
      const bool fits = there && sum <= p.x_rows;
      const int count = __popc(__ballot_sync(0xFFFFFFFFu, fits));
      if (fits) {
        sh.unit[lane] = u;
        if (kNv)  // an empty sum is zero, whatever the scale
          sh.unit_inverse[lane] = p.K > 0 && MXFP4_IN_BOUNDS(p, kDbgGlobal, p.global_scales + u.e, 4)
                                      ? 1.0f / __ldg(p.global_scales + u.e)
                                      : 1.0f;
      }
      if (lane == count - 1) {
        sh.n_units = count;
        sh.n_rows = sum;
      }
      if (lane < kMaxUnits) sh.unit_max[lane] = 15u;
      if (lane == 0) sh.far = 0;
    }
    __syncthreads();
    const int n_rows = sh.n_rows;
    int end = static_cast<int>(min(static_cast<int64_t>(last), static_cast<int64_t>(u0 + sh.n_units) * p.tiles));
    if (p.panels > 1) end = min(end, at + p.batch);
    const int n_tiles = end - at, total = n_tiles * n;
    const int f0 = total * warp / kWarps, f1 = total * (warp + 1) / kWarps;
    if (threadIdx.x < n_rows) {
      int i = 0;
      while (i + 1 < sh.n_units && sh.unit[i + 1].x <= static_cast<int>(threadIdx.x)) ++i;
      const int r = threadIdx.x - sh.unit[i].x;
      int64_t src = -1;
      if (r < sh.unit[i].n) {
        src = sh.unit[i].row0 + r;
        if (p.row_index != nullptr) src = index_at(p, src);
      }
      sh.x_row[threadIdx.x] = src >= 0 && src < p.src_rows ? src : -1;
      sh.x_unit[threadIdx.x] = r < sh.unit[i].n ? i : -1;
      sh.x_max[threadIdx.x] = 0u;
      sh.x_min[threadIdx.x] = 0xFFFFu;
    }

    // ---- x: copied in 16-byte pieces, four to a 32-element block, and scaled to
    // halves in place below.  With fewer rows than warps, several warps share one.
    // It goes before the weights, so that its scaling runs beside their first
    // copies (7168 x 7168 by 4 tokens: 14.4 -> 13.3 us), but after them where a
    // warp has one stage at most; x is then scaled by block, without the pass for
    // the rows' largest (2048 x 768 by 1 token: 5.6 -> 5.4 us; with the 3 stages of
    // experts' 1536 x 2048 by 1 token it took 10.0 -> 10.8).
    const int sharing = max(kWarps / n_rows, 1), rows_at_once = kWarps / sharing;
    const int my_row = warp / sharing < rows_at_once ? warp / sharing : n_rows;
    const int my_piece = (warp % sharing) * 32 + lane;
    auto copy_x = [&](int lo, int pieces) {
      for (int r = my_row; r < n_rows; r += rows_at_once) {
        const int64_t row = sh.x_row[r];
        const uint8_t* const src = p.x + ((row < 0 ? 0 : row) * p.ldx + lo * kChunk) * 2;
        const int there = row < 0 ? 0 : (p.K - lo * kChunk) / 8;  // pieces that x has
        const uint32_t to = smem_u32(x_s + r * p.x_pitch);
        for (int i = my_piece; i < pieces; i += sharing * 32) {
          const bool take = i < there && MXFP4_IN_BOUNDS(p, kDbgX, src + i * 16, 16);
          cp_async<16>(to + i * 16, take ? src + i * 16 : p.x, take ? 16 : 0);
        }
      }
      cp_commit();
    };
    if (!p.few) {
      __syncthreads();
      copy_x(0, min(n, p.chunks) * kBlocks * 4);
    }

    // ---- copies.  Row i of a tile is row tile_base + 32 * (i / 4) + i % 4 of the
    // weights; a copy takes the four rows of a quarter, eight lanes to a row's
    // 128 bytes.
    const int copy_row = lane >> 3, copy_at = (lane & 7) * 16;
    const int64_t quarter = 32 * static_cast<int64_t>(p.K >> 1);  // bytes of 32 rows
    Cursor in;
    in.panel = 0;
    in.f = f0;
    bool more = true;
    auto open_run = [&]() {  // the next run of chunks that is not empty
      for (;;) {
        if (in.f >= f1) {
          if (++in.panel >= p.panels) {
            more = false;
            return;
          }
          in.f = f0;
          continue;
        }
        const int t = in.f / n, first = in.f - t * n, len = min(f1 - in.f, n - first);
        in.f += len;
        in.chunk = in.panel * n + first;
        in.left = min(len, p.chunks - in.chunk);  // the last panel may be shorter
        if (in.left <= 0) continue;
        const int all_tile = tile0 + t, i = all_tile / p.tiles, tile = all_tile - i * p.tiles;
        const int e = sh.unit[i].e;
        const int base = (tile >> 3) * 128 + (tile & 7) * 4 + copy_row;
        in.quarters = base < p.N ? min(4, (p.N - base + 31) >> 5) : 0;
        in.whole = !p.half_rows && __all_sync(0xFFFFFFFFu, in.quarters == 4);
        in.row = p.codes + e * p.expert_codes + (in.quarters ? base : 0) * static_cast<int64_t>(p.K >> 1) + copy_at +
                 in.chunk * (kChunk / 2);
        in.scale = p.scales + e * p.expert_scales + (tile & 7) * 64 +
                   (static_cast<int64_t>(tile >> 3) * p.nKT + in.chunk * kChunkKt + (lane >> 2)) * kChunkBytes +
                   (lane & 3) * 16;
        return;
      }
    };
    open_run();
    uint32_t in_at = ring;  // the stage to fill
    const uint32_t copy_to = copy_row * kRowPitch + copy_at, ring_end = ring + ring_bytes;
    auto issue = [&]() {
      if (more) {
        const uint32_t to = in_at + copy_to, scale_to = in_at + kStageCodes + lane * 16;
        const uint8_t* row = in.row;
        const uint8_t* const scale = in.scale;
        in.row += kChunk / 2;
        in.scale += kChunkKt * kChunkBytes;
        if (in.whole && in.chunk != tail) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cp_async16_ahead(to + i * 4 * kRowPitch, row, MXFP4_IN_BOUNDS(p, kDbgCodes, row, 16) ? 16 : 0);
            row += quarter;
          }
          cp_async16_if(scale_to, scale,
                        lane < kScaleBytes / 16 && MXFP4_IN_BOUNDS(p, kDbgScales, scale, 16));
        } else {
          // rows past N, the last, partial chunk, and rows that start at 8-byte
          // boundaries
          const int k = in.chunk * kChunk + copy_at * 2;
          for (int i = 0; i < 4; ++i) {
            if (!p.half_rows) {
              const bool ok = i < in.quarters && k < p.K && MXFP4_IN_BOUNDS(p, kDbgCodes, row, 16);
              cp_async<16>(to + i * 4 * kRowPitch, ok ? row : p.codes, ok ? 16 : 0);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const bool ok =
                    i < in.quarters && k + 16 * h < p.K && MXFP4_IN_BOUNDS(p, kDbgCodes, row + 8 * h, 8);
                cp_async<8>(to + i * 4 * kRowPitch + 8 * h, ok ? row + 8 * h : p.codes, ok ? 8 : 0);
              }
            }
            row += quarter;
          }
          if (lane < kScaleBytes / 16) {
            // A piece is four rows' words of four columns.  The layout pads the columns to
            // a multiple of four with bytes that may be anything: zeros take their place
            // (32 experts' 5760 x 2880 by 64 tokens 82.4 -> 83.6 us).
            const int kt = in.chunk * kChunkKt + (lane >> 2);
            const bool ok = kt < p.nKT && MXFP4_IN_BOUNDS(p, kDbgScales, scale, 16);
            const int cols = p.K / (kNv ? 16 : 32) - 4 * kt;
            if (ok && cols < 4) {
#pragma unroll 1
              for (int i = 0; i < 4; ++i) cp_async4(scale_to + 4 * i, scale + 4 * i, cols);
            } else {
              cp_async<16>(scale_to, ok ? scale : p.scales, ok ? 16 : 0);
            }
          }
        }
        in_at += kStage;
        if (in_at == ring_end) in_at = ring;
        ++in.chunk;
        if (--in.left == 0) open_run();
      }
      cp_commit();  // an empty group at the end keeps the count of groups
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue();

    // a tile's sums of this lane (rows g and g + 8, columns 2c and 2c + 1 of
    // each block of 8) to y
    auto store = [&](int all_tile, const float (&acc)[NT][4]) {
      const int i = all_tile / p.tiles, tile = all_tile - i * p.tiles;
      const UnitRows u = sh.unit[i];
      const int row0 = (tile >> 3) * 128 + (tile & 7) * 4 + 32 * (g >> 2) + (g & 3);
      const float by = kNv ? sh.unit_inverse[i] : 1.0f;
      const int64_t size = p.y_f32 ? 4 : 2, ld = p.ldy * size;
      uint8_t* const to = p.y + (static_cast<int64_t>(u.row0) + 2 * c) * ld + row0 * size;
      const bool in_n[2] = {row0 < p.N, row0 + 64 < p.N};
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (k * 8 + 2 * c + e >= u.n) continue;
          uint8_t* const y = to + (k * 8 + e) * ld;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!in_n[h]) continue;
            const float v = kNv ? acc[k][2 * h + e] * by : acc[k][2 * h + e];
            if (p.y_f32) {
              float* q = reinterpret_cast<float*>(y) + 64 * h;
              if (MXFP4_IN_BOUNDS(p, kDbgY, q, 4)) *q = v;
            } else {
              uint16_t* q = reinterpret_cast<uint16_t*>(y) + 64 * h;
              if (MXFP4_IN_BOUNDS(p, kDbgY, q, 2))
                *q = static_cast<uint16_t>(kF16 ? pack_f16x2(v, 0.0f) : cvt_bf16x2(v, 0.0f));
            }
          }
        }
    };
    // sums of this lane in a slot of shared memory
    auto slot_at = [&](int slot) { return part_s + slot * (NT * 32) + lane; };

    uint32_t out_at = ring;  // the stage to read
    for (int panel = 0; panel < max(p.panels, 1); ++panel) {
      const int lo = panel * n, n_here = min(n, p.chunks - lo);  // this panel's chunks
      const int pieces = n_here * kBlocks * 4;
      if (panel > 0 || p.few) {
        if (threadIdx.x < n_rows) {
          sh.x_max[threadIdx.x] = 0u;
          sh.x_min[threadIdx.x] = 0xFFFFu;
        }
        __syncthreads();
        copy_x(lo, pieces);
        cp_wait<0>();
      } else {
        cp_wait<kStages>();  // all but the ring
      }
      bool by_row = true;  // one power of two for a row's whole panel of x
      if constexpr (!kF16) {
        by_row = !p.few;
        if (!p.few) {
          // A lane reads what it copied.  With the sign bits set, the order of the
          // patterns is that of the magnitudes; one less, zero is the largest.
          for (int r = my_row; r < n_rows; r += rows_at_once) {
            uint32_t most = 0x80008000u, least = 0xFFFFFFFFu;
            for (int i = my_piece; i < pieces; i += sharing * 32) {
              const uint4 v = *reinterpret_cast<const uint4*>(x_s + r * p.x_pitch + i * 16);
              const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t m = q[k] | 0x80008000u;
                most = __vmaxu2(most, m);
                least = __vminu2(least, (m - 0x00010001u) ^ 0x80008000u);
              }
            }
            most = max(most & 0x7FFFu, (most >> 16) & 0x7FFFu);
            least = min(least & 0xFFFFu, least >> 16);
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            if (lane == 0) {
              atomicMax(&sh.x_max[r], most);
              atomicMin(&sh.x_min[r], least);
              if (!kNv && sh.x_unit[r] >= 0) atomicMax(&sh.unit_max[sh.x_unit[r]], most >> 7);
            }
          }
          __syncthreads();
          // One power of two for a row's whole (panel of) x if that loses nothing:
          // all of it within 2^32; else one for each 32 elements.  For MXFP4, whose
          // weights may be of any size, the unit's largest goes into the weights'
          // scales (so that the sums are of the result's size) and its other rows
          // are within 2^8 of it.
          if (threadIdx.x < n_rows) {
            const uint32_t most = sh.x_max[threadIdx.x], least = sh.x_min[threadIdx.x] + 1u;
            const int unit = max(sh.x_unit[threadIdx.x], 0);
            const uint32_t e_max = sh.unit_max[unit];
            const uint32_t e = most != 0u ? max(most >> 7, 15u) : e_max;  // a row of zeros takes any scale
            const bool near =
                most == 0u || (most < 0x7F80u && max(least >> 7, 1u) + 32 >= most >> 7 && (kNv || e + 8 >= e_max));
            float inverse;
            half_scale(kNv ? most : e_max << 7, inverse);
            sh.x_scale[threadIdx.x] = kNv ? inverse : near ? __uint_as_float((127u + e - e_max) << 23) : 1.0f;
            if (!kNv) sh.unit_scale[unit] = inverse;
            if (!near) sh.far = 1;
          }
          __syncthreads();
          by_row = sh.far == 0;
        }
        for (int r = my_row; r < n_rows; r += rows_at_once) {
          float inverse_whole;
          const float f_whole = half_scale(sh.x_max[r], inverse_whole);
          for (int base = my_piece - lane; base < pieces; base += sharing * 32) {  // pieces % 32 == 0
            uint4* to = reinterpret_cast<uint4*>(x_s + r * p.x_pitch + (base + lane) * 16);
            const uint4 v = *to;
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
            float f = f_whole;
            if (!by_row) {
              uint32_t m = 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k) m = max_finite_bf16x2(m, q[k]);
              m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
              m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
              float inverse;
              f = half_scale(m, inverse);
              if (c == 0) xs_s[((base + lane) >> 2) * p.x_rows + r] = inverse;
            }
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = pack_f16x2(__uint_as_float(q[k] << 16) * f, __uint_as_float(q[k] & 0xFFFF0000u) * f);
            *to = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
      __syncthreads();

      // ---- the warp's share, a tile's run of chunks at a time
      float acc[NT][4];
      // Sums of `len` stages from chunk `ch` of the panel; x scaled by block needs
      // a factor for each, and few tokens one block of columns.
      auto multiply = [&](int ch, int len, const UnitRows& u, [[maybe_unused]] float common, auto by_block,
                          auto columns) {
        constexpr bool kByBlock = decltype(by_block)::value;
        constexpr int kCols = decltype(columns)::value;  // blocks of 8 tokens
        // The last kHold of a stage's scale chunks, with their codes, are taken
        // to registers at once, so that the next copy into the stage runs beside
        // their products: as many as the tokens' registers leave room for.  (None
        // held: 64000 x 7168 NVFP4 by 16 tokens 72 -> 78 us, the experts' 1536 x 2048
        // by 64 47.6 -> 51; nothing lost or won by 1 token.)
        constexpr int kHold = kByBlock ? 0 : kCols == 2 && !kNv ? (kF16 ? 1 : 0) : kChunkKt;
        constexpr int kPerKt = kBlocks / kChunkKt;  // 32-element blocks of a scale chunk
        constexpr int kUnroll = kByBlock ? 1 : kPerKt, kUnrollKt = kHold > 0 ? kChunkKt : 1;
        // A token past the unit's last reads the last one's x: its column of the
        // product is not stored.
        uint32_t xa[kCols];
#pragma unroll
        for (int t = 0; t < kCols; ++t)
          xa[t] = smem_u32(x_s) + (u.x + min(t * 8 + g, u.n - 1)) * p.x_pitch + c * 16 + ch * (kChunk * 2);
        [[maybe_unused]] uint32_t sx = smem_u32(xs_s) + (ch * kBlocks * p.x_rows + u.x + 2 * c) * 4;
        for (int f = 0; f < len; ++f) {
          cp_wait<kStages - 1>();
          __syncwarp();  // the copies of all lanes are in
          const uint32_t st = out_at;
          out_at += kStage;
          if (out_at == ring_end) out_at = ring;
          const uint32_t wa = st + g * kRowPitch + c * 4;
          // scale words of rows g and g + 8
          const uint32_t sa = st + kStageCodes + (g & 3) * 16 + (g >> 2) * 4;
          [[maybe_unused]] uint32_t words[2][kHold * kPerKt + 1], scale_words[2][kHold + 1];
          [[maybe_unused]] float run[kCols][4];  // NVFP4: sums of the whole stage
          if constexpr (kNv && !kByBlock) {
#pragma unroll
            for (int t = 0; t < kCols; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) run[t][i] = 0.0f;
          }
#pragma unroll kUnrollKt
          for (int kt = 0; kt < kChunkKt; ++kt) {
            constexpr int kFree = kChunkKt - kHold;
            if (kHold > 0 && kt == kFree) {
#pragma unroll
              for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int k = 0; k < kHold * kPerKt; ++k)
                  words[r][k] = lds32(wa + r * 8 * kRowPitch + (kFree * kPerKt + k) * 16);
#pragma unroll
                for (int k = 0; k < kHold; ++k) scale_words[r][k] = lds32(sa + r * 8 + (kFree + k) * 64);
              }
              __syncwarp();  // the stage is read
              issue();
            }
            const bool held = kHold > 0 && kt >= kFree;
            const uint32_t sw0 = held ? scale_words[0][kt - kFree] : lds32(sa + kt * 64);
            const uint32_t sw1 = held ? scale_words[1][kt - kFree] : lds32(sa + kt * 64 + 8);
#pragma unroll kUnroll
            for (int b4 = 0; b4 < kPerKt; ++b4) {
              const int b = kt * kPerKt + b4;
              uint32_t a0[4], a1[4];
              decode_word(held ? words[0][b - kFree * kPerKt] : lds32(wa + b * 16), a0);
              decode_word(held ? words[1][b - kFree * kPerKt] : lds32(wa + 8 * kRowPitch + b * 16), a1);
              [[maybe_unused]] float ws0 = 1.0f, ws1 = 1.0f;
              if constexpr (!kNv) {
                const uint32_t w0 = e8m0x2_to_bf16x2(sw0 >> (16 * (b4 / 2)));
                const uint32_t w1 = e8m0x2_to_bf16x2(sw1 >> (16 * (b4 / 2)));
                ws0 = __uint_as_float(b4 & 1 ? w0 & 0xFFFF0000u : w0 << 16);
                ws1 = __uint_as_float(b4 & 1 ? w1 & 0xFFFF0000u : w1 << 16);
                if constexpr (!kF16 && !kByBlock) {
                  ws0 *= common;
                  ws1 *= common;
                }
              } else {
                // lanes 0, 1 hold the block's first 16 elements, lanes 2, 3 the rest
                const uint32_t pick = (b4 * 2 + (c >> 1)) * 0x11u;  // that byte twice
                const uint32_t f0 = e4m3x2_to_f16x2(__byte_perm(sw0, 0u, pick));
                const uint32_t f1 = e4m3x2_to_f16x2(__byte_perm(sw1, 0u, pick));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  a0[i] = hmul2(a0[i], f0);
                  a1[i] = hmul2(a1[i], f1);
                }
              }
#pragma unroll
              for (int t = 0; t < kCols; ++t) {
                const uint4 xb = lds128(xa[t] + b * 64);
                if constexpr (kNv && !kByBlock) {
                  mma16816(run[t], a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
                  mma16816(run[t], a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
                } else {
                  float d[4];
                  mma16816_first(d, a0[0], a1[0], a0[1], a1[1], xb.x, xb.y);
                  mma16816(d, a0[2], a1[2], a0[3], a1[3], xb.z, xb.w);
                  float2 xs = make_float2(1.0f, 1.0f);
                  if constexpr (kByBlock) {
                    // columns past the unit's last read factors of other rows, inside x_rows
                    if (t * 8 + 2 * c < u.n) xs = lds64f(sx + (b * p.x_rows + t * 8) * 4);
                  }
                  if constexpr (kNv) {
                    acc[t][0] = fmaf(d[0], xs.x, acc[t][0]);
                    acc[t][1] = fmaf(d[1], xs.y, acc[t][1]);
                    acc[t][2] = fmaf(d[2], xs.x, acc[t][2]);
                    acc[t][3] = fmaf(d[3], xs.y, acc[t][3]);
                  } else {
                    acc[t][0] = fmaf(d[0], ws0 * xs.x, acc[t][0]);
                    acc[t][1] = fmaf(d[1], ws0 * xs.y, acc[t][1]);
                    acc[t][2] = fmaf(d[2], ws1 * xs.x, acc[t][2]);
                    acc[t][3] = fmaf(d[3], ws1 * xs.y, acc[t][3]);
                  }
                }
              }
            }
          }
          if constexpr (kNv && !kByBlock) {
#pragma unroll
            for (int t = 0; t < kCols; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[t][i] += run[t][i];
          }
          if constexpr (kHold == 0) {
            __syncwarp();  // the stage is read
            issue();
          }
#pragma unroll
          for (int t = 0; t < kCols; ++t) xa[t] += kChunk * 2;
          if constexpr (kByBlock) sx += kBlocks * p.x_rows * 4;
        }
      };
      for (int f = f0; f < f1;) {
        const int t = f / n, first = f - t * n, whole = min(f1 - f, n - first);
        f += whole;
        const int i = (tile0 + t) / p.tiles;
        const UnitRows u = sh.unit[i];
#pragma unroll
        for (int k = 0; k < NT * 4; ++k) acc[k >> 2][k & 3] = 0.0f;
        const int len = min(whole, n_here - first);
        if (len > 0) {
          const float common = kF16 || kNv ? 1.0f : sh.unit_scale[i];
          if (!kF16 && !by_row) {
            multiply(first, len, u, 1.0f, std::true_type{}, std::integral_constant<int, NT>{});
          } else if (NT == 2 && u.n <= 8) {
            multiply(first, len, u, common, std::false_type{}, std::integral_constant<int, 1>{});
          } else {
            multiply(first, len, u, common, std::false_type{}, std::integral_constant<int, NT>{});
          }
          if (!kF16 && by_row) {
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              if (k * 8 + 2 * c >= u.n) break;
              const float2 xs = *reinterpret_cast<const float2*>(&sh.x_scale[u.x + k * 8 + 2 * c]);
              acc[k][0] *= xs.x;
              acc[k][1] *= xs.y;
              acc[k][2] *= xs.x;
              acc[k][3] *= xs.y;
            }
          }
        }
        if (p.panels > 1) {
          // slot tile + warp: the shares are consecutive, so no two parts have the
          // same; a lane adds up the panels of its own
          float4* q = slot_at(t + warp);
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const float4 v = panel > 0 ? q[k * 32] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            q[k * 32] = make_float4(v.x + acc[k][0], v.y + acc[k][1], v.z + acc[k][2], v.w + acc[k][3]);
          }
        } else if (whole == n) {
          store(tile0 + t, acc);  // the tile is this warp's alone
        } else {
          // the first run of a share that starts inside a tile, or its last
          float4* q = slot_at(2 * warp + (first == 0));
#pragma unroll
          for (int k = 0; k < NT; ++k) q[k * 32] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
        }
      }
      if (p.panels > 1) __syncthreads();  // x is read
    }
    __syncthreads();

    // ---- the tiles that are summed over warps, in the warps' order
    if (p.panels > 1) {
      for (int t = warp; t < n_tiles; t += kWarps) {
        float acc[NT][4] = {};
        const int w1 = share_of(t * n + n - 1, total);
        for (int w = share_of(t * n, total); w <= w1; ++w) {
          if (total * w / kWarps >= total * (w + 1) / kWarps) continue;
          const float4* q = slot_at(t + w);
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            acc[k][0] += q[k * 32].x;
            acc[k][1] += q[k * 32].y;
            acc[k][2] += q[k * 32].z;
            acc[k][3] += q[k * 32].w;
          }
        }
        store(tile0 + t, acc);
      }
    } else if (n == 0) {
      // no elements to sum
      for (int t = warp; t < n_tiles; t += kWarps) {
        float acc[NT][4] = {};
        store(tile0 + t, acc);
      }
    } else if (f0 < f1 && f0 % n != 0 && f1 >= (f0 / n + 1) * n) {
      // this warp has the last part of a tile that others begin
      const int t = f0 / n;
      float acc[NT][4] = {};
      for (int w = share_of(t * n, total); w <= warp; ++w) {
        const int start = total * w / kWarps;
        if (start >= total * (w + 1) / kWarps) continue;
        const float4* q = slot_at(2 * w + (start <= t * n));
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          acc[k][0] += q[k * 32].x;
          acc[k][1] += q[k * 32].y;
          acc[k][2] += q[k * 32].z;
          acc[k][3] += q[k * 32].w;
        }
      }
      store(tile0 + t, acc);
    }
    at = end;
  }
}

constexpr int kMaxSmem = 227 * 1024 - 5 * 1024;  // dynamic; the rest holds Shared

template <bool kNv, bool kF16>
cudaError_t launch_typed(MatvecParams p, int64_t expected_units, int nt, cudaStream_t stream) {
  const auto kernel = nt == 1 ? matvec_kernel<kNv, kF16, 1> : matvec_kernel<kNv, kF16, 2>;
  const int R = 8 * nt;
  const int kStage = kStageCodes + (kNv ? 256 : 128);
  const int sms = sm_count();
  // Tiles of a CTA, about.  Its phases are few if x of all their units fits; x
  // too long to fit whole goes in panels, with sums for all tiles of a phase.
  const int64_t per_cta = (expected_units * p.tiles + sms - 1) / sms;
  const int unit_rows = static_cast<int>(p.rows < R ? (p.rows > 0 ? p.rows + (p.rows & 1) : 2) : R);
  const int slot_bytes = nt * 32 * 16;  // a tile's sums, 16 bytes to a lane and column block
  const int pitch_of_chunk = kChunk * 2, xs_of_chunk = kF16 ? 0 : kBlocks * 4;
  int64_t spanned = per_cta / (p.tiles > 0 ? p.tiles : 1) + 2;  // units that a CTA's tiles meet
  if (p.offsets == nullptr && spanned > expected_units) spanned = expected_units;
  const int free_bytes = kMaxSmem - kWarps * kStages * kStage;
  // whole: two slots per warp, and as many rows as there is room and use for
  const int row_bytes = p.chunks * (pitch_of_chunk + xs_of_chunk) + 64;
  const int64_t fit = (free_bytes - 2 * kWarps * slot_bytes) / row_bytes & ~1;
  if (fit >= unit_rows) {
    const int64_t use = spanned * unit_rows < kMaxRows ? spanned * unit_rows : kMaxRows;
    p.panels = p.chunks > 0 ? 1 : 0;
    p.panel = p.chunks;
    p.batch = 0;
    p.x_rows = static_cast<int32_t>(fit < use ? fit : use);
  } else {
    int64_t fewest = -1;
    for (int64_t n_batches = 1; n_batches <= (per_cta > 1 ? per_cta : 1) && (n_batches <= 64 || fewest < 0);
         ++n_batches) {
      const int64_t tiles = ((per_cta > 1 ? per_cta : 1) + n_batches - 1) / n_batches;
      const int64_t room = free_bytes - (tiles + kWarps) * slot_bytes - unit_rows * 64;
      const int64_t chunks = room / (unit_rows * (pitch_of_chunk + xs_of_chunk));
      if (chunks < 1) continue;
      int64_t panels = (p.chunks + chunks - 1) / chunks;
      if (panels < 2) panels = 2;  // there is room for the chunks, not for a whole x's slots
      if (fewest < 0 || n_batches * panels < fewest) {
        fewest = n_batches * panels;
        p.panels = static_cast<int32_t>(panels);
        p.panel = static_cast<int32_t>((p.chunks + panels - 1) / panels);
        p.batch = static_cast<int32_t>(tiles);
        p.x_rows = unit_rows;
      }
    }
  }
  p.few = per_cta * p.chunks <= kWarps;
  p.x_pitch = p.panel * pitch_of_chunk + 64;
  const int smem = kWarps * kStages * kStage + p.x_rows * (p.x_pitch + p.panel * xs_of_chunk) +
                   (p.panels > 1 ? p.batch + kWarps : 2 * kWarps) * slot_bytes;
  static std::atomic<uint64_t> ready[2];  // devices on which each kernel may use kMaxSmem
  if (const cudaError_t e = allow_smem(kernel, kMaxSmem, ready[nt - 1]); e != cudaSuccess) return e;
  // a CTA per SM, each with its share of the tiles (the experts that have
  // rows are known on the device alone: rows bound their number)
  const int64_t most = (p.offsets ? p.rows : expected_units) * static_cast<int64_t>(p.tiles);
  const int64_t grid = most < sms ? (most > 0 ? most : 1) : sms;
  return launch_pdl(kernel, static_cast<unsigned>(grid), kThreads, smem, stream, p);
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
  p.rows = static_cast<int32_t>(a.rows);
  p.N = static_cast<int32_t>(a.N);
  p.K = static_cast<int32_t>(a.K);
  p.E = a.E;
  p.nKT = static_cast<int32_t>((a.K / (a.nvfp4 ? 16 : 32) + 3) / 4);
  p.tiles = static_cast<int32_t>((a.N + 127) / 128) * 8;
  p.chunks = static_cast<int32_t>((a.K + kChunk - 1) / kChunk);
  p.expert_codes = a.N * (a.K / 2);
  p.expert_scales = (a.N + 127) / 128 * p.nKT * kChunkBytes;
  p.y_f32 = a.y_f32;
  p.half_rows = a.K % 32 != 0;
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.dbg, kDbgX, a.x, a.src_rows > 0 ? ((a.src_rows - 1) * a.ldx + a.K) * 2 : 0);
  debug_range(p.dbg, kDbgCodes, a.codes, a.E * p.expert_codes);
  debug_range(p.dbg, kDbgScales, a.scales, a.E * p.expert_scales);
  debug_range(p.dbg, kDbgGlobal, a.global_scales, a.nvfp4 ? a.E * 4 : 0);
  debug_range(p.dbg, kDbgIndex, a.row_index, a.row_index ? a.rows * 4 : 0);
  debug_range(p.dbg, kDbgOffsets, a.offsets, a.offsets ? (static_cast<int64_t>(a.E) + 1) * 4 : 0);
  debug_range(p.dbg, kDbgStatus, a.status, a.status ? 4 : 0);
  debug_range(p.dbg, kDbgY, a.y, a.rows > 0 ? ((a.rows - 1) * a.ldy + a.N) * (a.y_f32 ? 4 : 2) : 0);
#endif
  // Tokens per unit: 8 or 16 columns of the tensor-core product (more would
  // leave x no room).  16 read the weights once where 8 read them twice: 64000 x
  // 7168 NVFP4 by 16 tokens 72 us against 95; the experts' 2048 x 768 by 128
  // tokens, 8 rows to a segment, 34 against 38.  Fewer rows cost the registers for
  // nothing: 1536 x 2048 by 64 tokens, 4 rows to a segment, 52 against 47.6.
  // Segments whose average is near 8 have some longer.
  const int64_t avg = a.offsets ? (a.rows + a.E - 1) / (a.E > 0 ? a.E : 1) : a.rows;
  const int nt = avg <= (a.offsets ? 6 : 8) ? 1 : 2;
  const int64_t used = a.offsets ? (a.rows < a.E ? a.rows : a.E) : 1;  // segments with rows, about
  const int64_t units = a.offsets ? used : (a.rows + 8 * nt - 1) / (8 * nt);
  if (a.nvfp4)
    return a.f16 ? launch_typed<true, true>(p, units, nt, stream)
                 : launch_typed<true, false>(p, units, nt, stream);
  return a.f16 ? launch_typed<false, true>(p, units, nt, stream)
               : launch_typed<false, false>(p, units, nt, stream);
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

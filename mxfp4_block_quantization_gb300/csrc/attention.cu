// attention.cu — attention of one query token per sequence over the paged
// 4-bit cache, for sm_103a.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j over the positions j in
//   [max(0, n - window), n) of each sequence, with k and v decoded from
//   MXFP4 (e2m1 * 2^(s-127)) or NVFP4 (e2m1 * e4m3(s) / g).
// One pass over the cache with a running maximum and sum per head in
// float32.
//
// What bounds it: the cache is read once for the query heads that share a kv
// head, so HBM does, if the SMs keep up with decoding about 45 values a
// clock.  Both products run on the tensor cores with the cache as the 16-row
// operand, so up to 8 query heads cost what one does:
//   scores  S^T [16 positions x 8 heads] = K [16 x D] Q^T, a position's codes
//           as they lie (a lane's word of 8 codes meets the same 8 elements
//           of q);
//   output  O^T [16 values of D x 8 heads] = V^T [16 x 16 positions] P^T:
//           ldmatrix transposes V's 16-bit groups of four codes, so a
//           register holds four codes of each of two positions.
// With more heads to a kv head a unit may have two such column blocks.
// The sums keep the heads in the same columns in both, so the softmax's
// rescaling needs no exchange.
//
// A warp works alone, with its own ring of copies: the steps (32 positions) of
// all units (a sequence, a kv head, 8 query heads) are one sequence of which
// every warp that the GPU holds has an even share, whatever the lengths.  A unit
// that spans warps is joined by a second kernel.  Short contexts have a cluster
// of CTAs to each unit instead, whose parts are joined in shared memory.
//
// Scales.  K, MXFP4: a power of two of any size, applied in float32 to the
// 32-element partial scores; NVFP4: e2m1 * e4m3 has at most 6 bits and is
// formed in halves, exactly.  V: a position's scales vary along the sum, so
// they go into the operands: NVFP4 into V; MXFP4 into P, relative to the
// largest scale that the warp has met in that 32-value block (an integer
// maximum, with the output rescaled when it grows; under 2^-24 of it a scale
// is zero).  P is formed at 2^12 times its size and rounded to a half there,
// so it has 11 bits down to 2^-26 of the warp's largest and is lost under
// 2^-37 (beside a position that dominates with a small value, the others are
// the output); the denominator's sum keeps it in float32.  2^12 is divided out
// of the sums at the end.
//
// Measured, 64 query heads on 8: 64 sequences of up to 8192 positions (head_dim
// 128, MXFP4, 445 MB of cache) 98 to 100 us, 4.5 TB/s.  A copy of the kernel without
// the products took 87, one without the second kernel 5 less: what is left to win is
// the copies' latency at a unit's start and the parts' way through L2, not arithmetic
// (the vector units that decode are busy for 57 % of the cycles; a decode of V
// without its byte permutes, half the multiplications of the scores and simpler
// addresses each changed the time by 1 % at most).  One sequence of 131072 38.3 us
// (head_dim 64, NVFP4: 28.4), of 700 6.4 us.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache_device.cuh"
#include "fragments.cuh"
#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"

namespace mxfp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;   // positions of a warp's step
// Stages of a warp's ring, and CTAs of an SM that it is made for.  A third stage
// is worth the fourth CTA where the copies bound the call (two stages at four
// CTAs: 8 sequences of 32768, head_dim 64, 36.9 -> 39.7 us; one of 131072, head_dim
// 128, 40.8 -> 42.6), but not with a cluster to each unit, whose few steps want the
// warps (64 of 1024 positions: 21.7 us, with three stages 26.6).
__host__ __device__ constexpr int stages_of(int blocks, bool cluster) { return cluster || blocks > 4 ? 2 : 3; }
__host__ __device__ constexpr int ctas_of(int blocks, bool cluster, int column_blocks) {
  if (column_blocks > 1) return blocks <= 2 ? 3 : 2;
  return (blocks <= 2 ? 5 : blocks <= 4 ? 4 : 2) - (cluster || blocks > 4 ? 0 : 1);
}
constexpr int kColumns = 8;  // query heads of a column block of the products
constexpr float kLag = 3.0f;  // log2: how far a warp's reference may lag behind its maximum
                              // (0: 64 sequences of 8192 99.1 -> 100.2 us)
constexpr float kRaise = 12.0f;  // log2: what P is raised by; with kLag inside a half
constexpr float kLower = 0x1p-12f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttentionParams {
  const uint8_t* __restrict__ q;
  const uint8_t* __restrict__ codes[2];
  const uint8_t* __restrict__ scales[2];
  const float* __restrict__ global_scales[2];
  const int32_t* __restrict__ page_table;
  const int32_t* __restrict__ seq_lens;
  uint8_t* __restrict__ out;
  float* __restrict__ lse;
  float* __restrict__ part_o;   // [slot, 8 heads, head_dim]
  float* __restrict__ part_ml;  // [slot, 8 heads, 2]: maximum (log2), sum
  int4* __restrict__ parts;     // [unit]: see Parts
  int32_t* __restrict__ bad;    // [warp]: met a page out of range
  int32_t* __restrict__ status;
  int64_t q_seq_stride;
  int64_t q_head_stride;
  int64_t table_stride;
  int64_t max_len;
  uint64_t scale_bytes;  // of keys, and of values
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;     // query heads of a kv head
  int32_t columns;   // query heads of a unit, 8 or 16
  int32_t chunks;    // units of a kv head
  int32_t workers;   // warps that share the positions; 0: a warp, or a cluster, per unit
  int32_t ctas;      // of a unit's cluster, or 0
  int32_t num_pages;
  int32_t page_size;
  int32_t head_dim;
  int32_t window;
  int32_t f16;
  float softmax_scale;
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
  struct {
    DebugRanges dbg;
  } more;  // of the second list below
#endif
};

enum : int { kDbgQ = 0, kDbgCodes0, kDbgCodes1, kDbgScales0, kDbgScales1, kDbgTable, kDbgOut, kDbgPart };
enum : int { kDbgLens = 0, kDbgLse, kDbgStatus };

// The positions [lo, hi) of sequence b; a length out of range gives none.
__device__ __forceinline__ bool positions(const AttentionParams& p, int b, int& lo, int& hi) {
  const int32_t* at = p.seq_lens + b;
  const int n = MXFP4_IN_BOUNDS(p.more, kDbgLens, at, 4) ? __ldg(at) : 0;
  const bool ok = n >= 0 && n <= p.max_len;
  hi = ok ? n : 0;
  lo = p.window > 0 && hi > p.window ? hi - p.window : 0;
  return ok;
}
__device__ __forceinline__ int steps_of(const AttentionParams& p, int b) {
  int lo, hi;
  positions(p, b, lo, hi);
  return static_cast<int>((static_cast<unsigned>(hi - lo) + kStep - 1) / kStep);
}
__device__ __forceinline__ bool one_sequence(const AttentionParams& p) {
  return p.num_seqs == 1 && p.workers >= p.num_kv_heads * p.chunks;
}
// A single sequence's units are padded to whole shares, so that no warp has
// parts of two (32768 positions, 8 heads: 18.6 -> 17.5 us); with several sequences
// of any lengths a share may end anywhere.
__device__ __forceinline__ int padded_steps(const AttentionParams& p, int steps, int share) {
  return one_sequence(p) ? (steps + share - 1) / share * share : steps;
}
// Steps of one warp, from the steps of all units.
__device__ __forceinline__ int share_of(const AttentionParams& p, int& total, int units) {
  if (one_sequence(p)) {
    const int steps = total / units, per_unit = p.workers / units;
    const int share = max((steps + per_unit - 1) / per_unit, 1);
    total = padded_steps(p, steps, share) * units;
    return share;
  }
  return max((total + p.workers - 1) / p.workers, 1);
}
// The steps of all units, and their prefix sums by thread.
__device__ __forceinline__ int scan_steps(const AttentionParams& p, int units, int* prefix) {
  __shared__ int warp_sum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b < p.num_seqs) sum += steps_of(p, b) * units;
  }
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, sum, k);
    if (lane >= k) sum += v;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) sum += warp_sum[w];
    total += warp_sum[w];
  }
  prefix[threadIdx.x] = sum;
  __syncthreads();
  return total;
}
// The sequence that step `at` belongs to, and its first step.
__device__ __forceinline__ int find_sequence(const AttentionParams& p, const int* prefix, int units,
                                             int at, int& first) {
  first = 0;
  if (p.num_seqs == 1) return 0;
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] > at) hi = mid; else lo = mid + 1;
  }
  if (lo > 0) first = prefix[lo - 1];
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  int b = lo * per;
  for (;; ++b) {
    const int n = steps_of(p, b) * units;
    if (at < first + n || b + 1 >= p.num_seqs) return b;
    first += n;
  }
}

// Who holds the parts of a unit: the warps first..last, but of CTAs cta0..cta1 - 1,
// which have no other unit, the first warp for all.
struct Parts {
  int first, last, cta0, cta1;
  __device__ __forceinline__ int count() const {
    return last - first + 1 - max(cta1 - cta0, 0) * (kWarps - 1);
  }
  __device__ __forceinline__ int warp(int k) const {
    const int before = kWarps * cta0 - first, whole = max(cta1 - cta0, 0);
    if (whole == 0 || k < before) return first + k;
    return k < before + whole ? kWarps * (cta0 + k - before) : first + k + whole * (kWarps - 1);
  }
};
__device__ __forceinline__ Parts parts_of(int unit_at, int steps, int share) {
  Parts r;
  r.first = unit_at / share;
  r.last = (unit_at + steps - 1) / share;
  r.cta0 = (r.first * share == unit_at ? r.first + kWarps - 1 : r.first + kWarps) / kWarps;
  r.cta1 = ((r.last + 1) * share == unit_at + steps ? r.last + 1 : r.last) / kWarps;
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// kN consecutive float32 of shared memory, kN * 4-byte aligned.
template <int kN>
__device__ __forceinline__ void lds_floats(float (&f)[kN], uint32_t a) {
  if constexpr (kN % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
      const uint4 v = lds128(a + 16 * i);
      f[4 * i] = __uint_as_float(v.x);
      f[4 * i + 1] = __uint_as_float(v.y);
      f[4 * i + 2] = __uint_as_float(v.z);
      f[4 * i + 3] = __uint_as_float(v.w);
    }
  } else if constexpr (kN % 2 == 0) {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      const float2 v = lds64f(a + 8 * i);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = __uint_as_float(lds32(a + 4 * i));
  }
}

// Status word of a call without shared steps: every length and every page that a
// sequence needs.  `per` threads to a sequence; four entries of four sequences in
// flight in each.
__device__ __forceinline__ void write_status(const AttentionParams& p) {
  constexpr int kSeqs = 4, kEntries = 4;
  int per = 1;
  while (per < kThreads && static_cast<int64_t>(kEntries * per) * p.page_size < p.max_len) per *= 2;
  const int lane = threadIdx.x % per, stride = kThreads / per;
  int bad = 0;
  for (int64_t b0 = threadIdx.x / per; b0 < p.num_seqs; b0 += kSeqs * stride) {
    int64_t i[kSeqs], last[kSeqs];
    int32_t page[kSeqs][kEntries];
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      const int64_t b = b0 + k * stride;
      i[k] = 0;
      last[k] = -1;
      if (b >= p.num_seqs) continue;
      int lo, hi;
      if (!positions(p, static_cast<int>(b), lo, hi)) bad = 1;
      i[k] = lo / p.page_size + lane;
      last[k] = hi > lo ? (hi - 1) / p.page_size : -1;
    }
    bool more = true;
    while (more) {
      more = false;
#pragma unroll
      for (int k = 0; k < kSeqs; ++k)
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
          const int64_t at = i[k] + j * per;
          const int32_t* entry = p.page_table + (b0 + k * stride) * p.table_stride + at;
          page[k][j] = at > last[k] ? 0 : MXFP4_IN_BOUNDS(p, kDbgTable, entry, 4) ? __ldg(entry) : -1;
        }
#pragma unroll
      for (int k = 0; k < kSeqs; ++k) {
#pragma unroll
        for (int j = 0; j < kEntries; ++j)
          if (i[k] + j * per <= last[k] && (page[k][j] < 0 || page[k][j] >= p.num_pages)) bad = 1;
        i[k] += kEntries * per;
        more |= i[k] <= last[k];
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && MXFP4_IN_BOUNDS(p.more, kDbgStatus, p.status, 4)) *p.status = bad ? -7 : 0;
}

// Shared memory of a stage, for head_dim = 32 * DB.
template <bool kNv, int DB>
struct Stage {
  static constexpr int kScale = kNv ? 2 * DB : DB;         // scale bytes of a position
  static constexpr int kWords = (kScale + 3) / 4;
  // Positions an odd number of 16-byte pieces apart: eight rows of a fragment
  // then lie in different banks.
  static constexpr int kPitch = (DB | 1) * 16;
  static constexpr int kK = 0;
  static constexpr int kV = kStep * kPitch;
  static constexpr int kScaleK = 2 * kStep * kPitch;
  // MXFP4: K's scales as float32 [position][block], V's as halves relative to
  // the running largest, [block][c][8 positions each][2] (a B fragment's
  // pairs); NVFP4: the bytes, [position][words] and [block][position].
  static constexpr int kScaleV = kScaleK + kStep * (kNv ? kWords * 4 : DB * 4);
  static constexpr int kValid = kScaleV + kStep * (kNv ? kWords * 4 : DB * 2);  // a bit per position
  // As they are copied: the 4-byte words that hold a position's scale bytes, of
  // K and of V, with the bytes before them in the first (when they can start
  // inside a word), and the page of the position two steps on.
  static constexpr int kRaw = kScale % 4 == 0 ? kWords : (kScale + (kScale % 2 == 0 ? 2 : 3) + 3) / 4;
  static constexpr int kRawK = kValid + 16;
  static constexpr int kRawV = kRawK + kStep * kRaw * 4;
  static constexpr int kSkip = kRawV + kStep * kRaw * 4;
  static constexpr int kPage = kSkip + (kScale % 4 == 0 ? 0 : kStep * 4);
  static constexpr int kBytes = kPage + kStep * 4;
};

// Four values of the output: acc / sum (zero without positions), NVFP4 with
// V's global scale divided out.
template <bool kNv>
__device__ __forceinline__ void store_out(const AttentionParams& p, int64_t head, int d, int D, float4 acc,
                                          float sum) {
  // one after the other: their product may be past float32
  const float by = kNv ? global_scale_or_one(p.global_scales[1]) : 1.0f;
  auto one = [&](float v) { return sum == 0.0f ? 0.0f : kNv ? v / sum / by : v / sum; };
  uint2 y;
  if (p.f16) {
    y.x = pack_f16x2(one(acc.x), one(acc.y));
    y.y = pack_f16x2(one(acc.z), one(acc.w));
  } else {
    y.x = cvt_bf16x2(one(acc.x), one(acc.y));
    y.y = cvt_bf16x2(one(acc.z), one(acc.w));
  }
  uint8_t* to = p.out + (head * D + d) * 2;
  if (MXFP4_IN_BOUNDS(p, kDbgOut, to, 8)) *reinterpret_cast<uint2*>(to) = y;
}
__device__ __forceinline__ void store_lse(const AttentionParams& p, int64_t head, float sum, float top) {
  if (p.lse != nullptr && MXFP4_IN_BOUNDS(p.more, kDbgLse, p.lse + head, 4))
    p.lse[head] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
}

// The scale bytes of this lane's position, as words that start with the first.
template <typename S>
__device__ __forceinline__ void own_scales(uint32_t (&k)[S::kWords], uint32_t (&v)[S::kWords], uint32_t st,
                                           int lane) {
  uint32_t a[S::kRaw + 1], b[S::kRaw + 1];
#pragma unroll
  for (int i = 0; i < S::kRaw; ++i) {
    a[i] = lds32(st + S::kRawK + (lane * S::kRaw + i) * 4);
    b[i] = lds32(st + S::kRawV + (lane * S::kRaw + i) * 4);
  }
  a[S::kRaw] = b[S::kRaw] = 0u;
  const uint32_t skip = S::kScale % 4 == 0 ? 0u : 8u * lds32(st + S::kSkip + lane * 4);
#pragma unroll
  for (int i = 0; i < S::kWords; ++i) {
    k[i] = S::kScale % 4 == 0 ? a[i] : __funnelshift_r(a[i], a[i + 1], skip);
    v[i] = S::kScale % 4 == 0 ? b[i] : __funnelshift_r(b[i], b[i + 1], skip);
  }
}

// The parts of a unit that the warps of a cluster, or of a CTA, hold in their
// rings, joined: each thread four values of a head, the parts read from the CTAs'
// shared memory kBatch at a time.  `store(head, quad, acc, sum, top)`.  (Each warp's
// part to the workspace instead: one sequence of 131072, head_dim 64, 28.3 -> 31.1 us.)
template <int DB, bool kCluster, int kHeads, typename Store>
__device__ __forceinline__ void join_rings(uint32_t rings, uint32_t ring_bytes, int ctas, int heads, Store store) {
  constexpr int D = 32 * DB, kQuads = D / 4, kBatch = kCluster ? 8 : kWarps;
  const int parts = ctas * kWarps;
  for (int u = (kCluster ? cluster_rank() : 0) * kThreads + threadIdx.x; u < heads * kQuads; u += ctas * kThreads) {
    const int h = u / kQuads, quad = u - h * kQuads;
    float top = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < parts; s0 += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int s = s0 + k;
        ml[k] = make_float2(-INFINITY, 0.0f);
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (s < parts) {
          uint32_t from = rings + (s % kWarps) * ring_bytes;
          if constexpr (kCluster) from = cluster_address(from, s / kWarps);
          ml[k] = ld_cluster_f2(from + (kHeads * D + h * 2) * 4);
          v[k] = ld_cluster_f4(from + (h * D + quad * 4) * 4);
        }
      }
      float x = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) x = fmaxf(x, ml[k].x);
      const float z = x == -INFINITY ? 0.0f : x;
      const float keep = exp2_approx(top - z);
      top = x;
      sum *= keep;
      acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = exp2_approx(ml[k].x - z);
        sum += ml[k].y * f;
        acc.x += v[k].x * f;
        acc.y += v[k].y * f;
        acc.z += v[k].z * f;
        acc.w += v[k].w * f;
      }
    }
    store(h, quad, acc, sum, top);
  }
}

template <bool kNv, int DB, bool kCluster, int NB>
__global__ void __launch_bounds__(kThreads, ctas_of(DB, kCluster, NB)) attention_kernel(const AttentionParams p) {
  constexpr int kHeads = NB * kColumns;
  constexpr int kStages = stages_of(DB, kCluster), kAhead = kStages - 1;
  using S = Stage<kNv, DB>;
  constexpr int D = 32 * DB;
  static_assert(kStages * S::kBytes >= kHeads * (D + 2) * 4, "a part fits in a warp's ring");
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  const int ctas = kCluster ? p.ctas : 1;  // of a unit
  if (p.workers == 0 && blockIdx.x >= gridDim.x - ctas && p.status != nullptr) {
    if (blockIdx.x == gridDim.x - 1) write_status(p);
    return;
  }
  // A unit of work is the positions of one sequence for one kv head and 8 of
  // its query heads, in steps of 32.
  const int units_per_seq = p.num_kv_heads * p.chunks;
  const int worker = kCluster ? cluster_rank() * kWarps + warp : blockIdx.x * kWarps + warp;
  __shared__ int prefix[kThreads];  // steps up to and with each thread's sequences
  int at = 0, end = 0, share = 1;   // this warp's steps, over all units
  if (kCluster) {
    end = 1;
  } else if (p.workers > 0) {
    int total = scan_steps(p, units_per_seq, prefix);
    share = share_of(p, total, units_per_seq);
    at = static_cast<int>(min(static_cast<int64_t>(share) * worker, static_cast<int64_t>(total)));
    end = min(total - at, share) + at;
  } else if (worker < static_cast<int64_t>(p.num_seqs) * units_per_seq) {
    end = 1;
  }
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kBytes;
  bool bad = false;  // shared steps: a page was out of range
  while (at < end) {
    // the unit that step `at` is in, and this warp's part of its steps
    int b, unit, s0 = 0, s1;
    bool whole = true;    // this warp has the whole unit
    bool joined = false;  // the CTA's warps have this unit alone, and join their parts
    if constexpr (kCluster) {
      const int which = blockIdx.x / ctas;
      b = which / units_per_seq;
      unit = which - b * units_per_seq;
      const int steps = steps_of(p, b), part = (steps + ctas * kWarps - 1) / (ctas * kWarps);
      s0 = min(steps, worker * part);
      s1 = min(steps, s0 + part);
      at = end;
    } else if (p.workers > 0) {
      int unit_at;
      b = find_sequence(p, prefix, units_per_seq, at, unit_at);
      const int steps = steps_of(p, b);
      const int padded = padded_steps(p, steps, share);
      unit = (at - unit_at) / padded;
      unit_at += unit * padded;
      s0 = at - unit_at;
      s1 = min(padded, s0 + (end - at));
      at += s1 - s0;
      const Parts parts = parts_of(unit_at, steps, share);
      const int cta = blockIdx.x;
      whole = parts.count() == 1;
      joined = cta >= parts.cta0 && cta < parts.cta1;
      int4* to = p.parts + static_cast<int64_t>(b) * units_per_seq + unit;
      if (s0 == 0 && lane == 0 && MXFP4_IN_BOUNDS(p, kDbgPart, to, 16))
        *to = make_int4(parts.first, parts.last, parts.cta0, parts.cta1);
      if (s0 >= steps) continue;  // padding
    } else {
      b = worker / units_per_seq;
      unit = worker - b * units_per_seq;
      s1 = steps_of(p, b);
      at = end;
    }
    const int kvh = unit % p.num_kv_heads, chunk = unit / p.num_kv_heads;
    int lo, hi;
    positions(p, b, lo, hi);
    // positions past the last one, up to 2^31 + a step and a share's padding, are unsigned
    const unsigned first = lo + static_cast<unsigned>(s0) * kStep;
    const unsigned last = min(static_cast<unsigned>(hi), lo + static_cast<unsigned>(s1) * kStep);
    const unsigned page_size = p.page_size;
    const int head0 = kvh * p.group + chunk * kHeads;
    const int heads = min(kHeads, p.group - chunk * kHeads);
    __syncwarp();  // the unit before is done with the ring

    // ---- copies
    const int32_t* table = p.page_table + b * p.table_stride;
    unsigned next = first + lane;  // this lane's position in the step to copy
    unsigned in_page = next % page_size;
    const unsigned page_step = kStep / page_size;
    const unsigned in_step = kStep - page_step * page_size;
    // where the position kAhead steps on has its page
    unsigned ahead = next + kAhead * kStep;
    unsigned ahead_at = ahead / page_size, ahead_in = ahead - ahead_at * page_size;
    auto load_page = [&](unsigned position) {
      const int32_t* entry = table + position / page_size;
      return position < last && MXFP4_IN_BOUNDS(p, kDbgTable, entry, 4) ? __ldg(entry) : -1;
    };
    uint32_t fill = 0;  // stage to fill
    auto issue = [&](int page) {
      if (next - lane < last) {
        const bool ok = next < last && page >= 0 && page < p.num_pages;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, ok);
        const uint32_t row = ok ? (static_cast<uint32_t>(page) * p.num_kv_heads + kvh) * page_size + in_page : 0u;
        const uint32_t st = ring + fill;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          const int piece = i * 32 + lane, to = piece / DB, ch = piece - to * DB;
          const uint64_t off = static_cast<uint64_t>(__shfl_sync(0xFFFFFFFFu, row, to)) * (D / 2) + ch * 16;
          const int take = (valid >> to) & 1u ? 16 : 0;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint8_t* src = p.codes[part] + off;
            cp_async<16>(st + (part ? S::kV : S::kK) + to * S::kPitch + ch * 16, src,
                         MXFP4_IN_BOUNDS(p, kDbgCodes0 + part, src, take) ? take : 0);
          }
        }
        // a position that is not there has zero scales: nothing of V, and its
        // scores are masked
        const uint64_t soff = static_cast<uint64_t>(row) * S::kScale;
        const int skip = S::kScale % 4 == 0 ? 0 : static_cast<int>(soff & 3);
#pragma unroll
        for (int i = 0; i < S::kRaw; ++i) {
          const uint64_t w = soff - skip + 4 * i;
          const int64_t left = static_cast<int64_t>(p.scale_bytes - w);
          const int take = !ok || (S::kScale % 4 != 0 && left <= 0) ? 0
                           : S::kScale % 4 != 0 && left < 4         ? static_cast<int>(left)
                                                                    : 4;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint8_t* src = p.scales[part] + (take ? w : 0);
            cp_async4(st + (part ? S::kRawV : S::kRawK) + (lane * S::kRaw + i) * 4, src,
                      MXFP4_IN_BOUNDS(p, kDbgScales0 + part, src, take) ? take : 0);
          }
        }
        if constexpr (S::kScale % 4 != 0) sts32(st + S::kSkip + lane * 4, skip);
        {
          const int32_t* entry = table + (ahead < last ? ahead_at : 0);
          cp_async4(st + S::kPage + lane * 4, entry,
                    ahead < last && MXFP4_IN_BOUNDS(p, kDbgTable, entry, 4) ? 4 : 0);
        }
        if (lane == 0) sts32(st + S::kValid, valid);
        fill = fill == kAhead * S::kBytes ? 0 : fill + S::kBytes;
        next += kStep;
        in_page += in_step;
        if (in_page >= page_size) in_page -= page_size;
        ahead += kStep;
        ahead_at += page_step;
        ahead_in += in_step;
        if (ahead_in >= page_size) {
          ahead_in -= page_size;
          ++ahead_at;
        }
      }
      cp_commit();  // an empty group at the end keeps the count of groups
    };
    {
      int page[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) page[i] = load_page(next + i * kStep);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) issue(page[i]);
    }

    // ---- q: a lane holds elements 8c..8c+7 of each 32-element block of head g,
    // as halves; BF16 scaled by the head's power of two (see matvec.cu), which keeps
    // it exactly down to 2^-32 of its largest element and to 2^-40 of that below.  (A
    // power for each block where a head is wider, applied to the blocks' partial
    // scores: 64 sequences of 8192 99.4 -> 101.9 us, one of 700 6.4 -> 6.7, 32 of 4096
    // with 128 heads on 8 49.6 -> 51.5, whether a head is or not.)  With MXFP4
    // keys, which may be of any size, the largest of the unit's heads goes into the
    // keys' scales, so that the scores' sums are of the size of q . k; not above 1, so
    // that a head of any size leaves the others' sums as they are.
    uint4 q[NB][DB];
    float qs[NB][2];  // what undoes it, with the softmax's scale, for heads 2c and 2c + 1 of a block
    float inverse[NB], common = 1.0f;
    auto set_factor = [&](int n, float more) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // not zero: a masked score is -infinity, and stays that; the smallest float
        // instead moves no score by more than 2^-21
        const float f = __shfl_sync(0xFFFFFFFFu, inverse[n], 8 * c + 4 * e) * fabsf(more);
        qs[n][e] = f == 0.0f ? 0x1p-149f : f;
      }
    };
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int h = n * kColumns + g;
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(p.q) + b * p.q_seq_stride +
                           static_cast<int64_t>(head0 + h) * p.q_head_stride + c * 8;
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        uint4& v = q[n][i];
        v = make_uint4(0u, 0u, 0u, 0u);
        if (h < heads && MXFP4_IN_BOUNDS(p, kDbgQ, qp + i * 32, 16))
          v = __ldg(reinterpret_cast<const uint4*>(qp + i * 32));
        m = max_finite_bf16x2(max_finite_bf16x2(m, v.x), v.y);
        m = max_finite_bf16x2(max_finite_bf16x2(m, v.z), v.w);
      }
      inverse[n] = 1.0f;
      if (!p.f16) {
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const float f = half_scale(m, inverse[n]);
        auto scaled = [&](uint32_t v) {
          return pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f);
        };
#pragma unroll
        for (int i = 0; i < DB; ++i)
          q[n][i] = make_uint4(scaled(q[n][i].x), scaled(q[n][i].y), scaled(q[n][i].z), scaled(q[n][i].w));
      }
      const float more = p.softmax_scale * kLog2e / (kNv ? global_scale_or_one(p.global_scales[0]) : 1.0f);
      const uint32_t sign = more < 0.0f ? 0x80008000u : 0u;  // a larger product is a larger score
#pragma unroll
      for (int i = 0; i < DB; ++i)
        q[n][i] = make_uint4(q[n][i].x ^ sign, q[n][i].y ^ sign, q[n][i].z ^ sign, q[n][i].w ^ sign);
      if constexpr (kNv) set_factor(n, more);
    }
    if constexpr (!kNv) {
      uint32_t bits = 1u << 23;  // the powers' order is that of their bits
#pragma unroll
      for (int n = 0; n < NB; ++n) bits = max(bits, __float_as_uint(inverse[n]));
      // (In every form tried 128 heads on 8, 32 of 4096, took 47.6 -> 49 us for this, at
      // 255 registers; 64 sequences of 8192 100 -> 99.)
      bits = min(__reduce_max_sync(0xFFFFFFFFu, bits), (127u - 15u) << 23);
      common = __uint_as_float(bits);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        inverse[n] *= __uint_as_float((254u << 23) - bits);
        set_factor(n, p.softmax_scale * kLog2e);
      }
    }

    float m[NB][2], l[NB][2];  // of heads 2c and 2c + 1 of a block, log2
    float o[NB][DB][2][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[n][i][j >> 2][j & 3] = 0.0f;
    }
    int vref[DB];  // MXFP4: the largest scale byte of V so far, per block (same in all lanes)
#pragma unroll
    for (int i = 0; i < DB; ++i) vref[i] = 0;

    uint32_t read = 0;
    for (unsigned t0 = first; t0 < last; t0 += kStep) {
      cp_wait<kAhead - 1>();
      const uint32_t st = ring + read;
      read = read == kAhead * S::kBytes ? 0 : read + S::kBytes;
      // a lane has copied its position's scales: what all lanes need of them, once
      {
        uint32_t sk[S::kWords], sv[S::kWords];
        own_scales<S>(sk, sv, st, lane);
        if constexpr (kNv) {
#pragma unroll
          for (int i = 0; i < S::kWords; ++i) sts32(st + S::kScaleK + (lane * S::kWords + i) * 4, sk[i]);
#pragma unroll
          for (int i = 0; i < S::kScale; ++i)
            sts8(st + S::kScaleV + i * kStep + lane, sv[i / 4] >> (8 * (i % 4)));
        } else {
          int byte[DB];
          bool more = false;
#pragma unroll
          for (int i = 0; i < DB; ++i) {
            const uint32_t pair = e8m0x2_to_bf16x2(sk[i / 4] >> (16 * (i / 2 % 2)));
            const float f = __uint_as_float(i & 1 ? pair & 0xFFFF0000u : pair << 16) * common;
            sts32(st + S::kScaleK + (lane * DB + i) * 4, __float_as_uint(f));
            byte[i] = static_cast<int>((sv[i / 4] >> (8 * (i % 4))) & 0xFFu);
            more |= byte[i] > vref[i];
          }
          if (__any_sync(0xFFFFFFFFu, more)) {
#pragma unroll
            for (int i = 0; i < DB; ++i) {
              const int now = static_cast<int>(
                  __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(max(byte[i], vref[i]))));
              const float f = __uint_as_float(static_cast<uint32_t>(max(127 + vref[i] - now, 0)) << 23);
              vref[i] = now;
#pragma unroll
              for (int j = 0; j < 8 * NB; ++j) o[j >> 3][i][(j >> 2) & 1][j & 3] *= f;
            }
          }
          const uint32_t to = st + S::kScaleV + ((lane & 7) >> 1) * 16 + (lane >> 3) * 4 + (lane & 1) * 2;
#pragma unroll
          for (int i = 0; i < DB; ++i) {  // 2^(byte - vref), down to the smallest half
            const float f = __uint_as_float(static_cast<uint32_t>(max(127 + byte[i] - vref[i], 0)) << 23);
            sts16(to + i * 64, pack_f16x2(f, 0.0f));
          }
        }
      }
      const int next_page = static_cast<int>(lds32(st + S::kPage + lane * 4));
      __syncwarp();  // all lanes' copies and scales are in; the stage read last is free
      issue(next_page);
      const uint32_t valid = lds32(st + S::kValid);

      // ---- scores of 2 x 16 positions by 8 heads of each block
      float s[NB][2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4 * NB; ++i) s[i >> 2][t][i & 3] = 0.0f;
        uint32_t w0[S::kWords], w1[S::kWords];  // scales of positions g and g + 8
        float f0[DB], f1[DB];
        if constexpr (kNv) {
#pragma unroll
          for (int i = 0; i < S::kWords; ++i) {
            w0[i] = lds32(st + S::kScaleK + ((t * 16 + g) * S::kWords + i) * 4);
            w1[i] = lds32(st + S::kScaleK + ((t * 16 + g + 8) * S::kWords + i) * 4);
          }
        } else {
          lds_floats<DB>(f0, st + S::kScaleK + (t * 16 + g) * DB * 4);
          lds_floats<DB>(f1, st + S::kScaleK + (t * 16 + g + 8) * DB * 4);
        }
        const uint32_t ka = st + S::kK + (t * 16 + g) * S::kPitch + c * 4;
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          uint32_t a0[4], a1[4];
          decode_word(lds32(ka + i * 16), a0);
          decode_word(lds32(ka + 8 * S::kPitch + i * 16), a1);
          if constexpr (kNv) {
            const uint32_t pick = ((i & 1) * 2 + (c >> 1)) * 0x11u;  // the block's byte, twice
            const uint32_t e0 = e4m3x2_to_f16x2(__byte_perm(w0[i / 2], 0u, pick));
            const uint32_t e1 = e4m3x2_to_f16x2(__byte_perm(w1[i / 2], 0u, pick));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a0[k] = hmul2(a0[k], e0);
              a1[k] = hmul2(a1[k], e1);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              mma16816(s[n][t], a0[0], a1[0], a0[1], a1[1], q[n][i].x, q[n][i].y);
              mma16816(s[n][t], a0[2], a1[2], a0[3], a1[3], q[n][i].z, q[n][i].w);
            }
          } else {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              float d[4];
              mma16816_first(d, a0[0], a1[0], a0[1], a1[1], q[n][i].x, q[n][i].y);
              mma16816(d, a0[2], a1[2], a0[3], a1[3], q[n][i].z, q[n][i].w);
              s[n][t][0] = fmaf(d[0], f0[i], s[n][t][0]);
              s[n][t][1] = fmaf(d[1], f0[i], s[n][t][1]);
              s[n][t][2] = fmaf(d[2], f1[i], s[n][t][2]);
              s[n][t][3] = fmaf(d[3], f1[i], s[n][t][3]);
            }
          }
        }
      }
      if (valid != 0xFFFFFFFFu) {  // the last step, or a page that is not there
        bad |= valid != (last - t0 < kStep ? (1u << (last - t0)) - 1u : 0xFFFFFFFFu);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (((valid >> (t * 16 + g + 8 * r)) & 1u) == 0u) {
#pragma unroll
              for (int n = 0; n < NB; ++n) s[n][t][2 * r] = s[n][t][2 * r + 1] = -INFINITY;
            }
      }

      // ---- running maximum and sum.  The reference m may lag behind the
      // maximum by kLag (P then grows to 2^(kRaise + kLag) at most, inside a half),
      // so that the output is rescaled a few times at all, not at every new maximum.
      float x[NB][2];
      bool far = false;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = fmaxf(fmaxf(s[n][0][e], s[n][0][2 + e]), fmaxf(s[n][1][e], s[n][1][2 + e])) * qs[n][e];
          far |= x[n][e] > m[n][e] + kLag;
        }
      if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = x[n][e];
#pragma unroll
            for (int k = 4; k < 32; k *= 2) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, k));
            y = fmaxf(y, m[n][e]);
            const float keep = exp2_approx(m[n][e] - (y == -INFINITY ? 0.0f : y));
            m[n][e] = y;
            l[n][e] *= keep;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[n][i][j >> 1][(j & 1) * 2 + e] *= keep;
          }
      }
      uint32_t pt[NB][2][2];  // P^T of each block: columns of heads, pairs of positions
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float z0 = (m[n][0] == -INFINITY ? 0.0f : m[n][0]) - kRaise;
        const float z1 = (m[n][1] == -INFINITY ? 0.0f : m[n][1]) - kRaise;
        uint32_t pk[2][2];  // 2^kRaise * P of positions g and g + 8 of each half, heads 2c and 2c + 1
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float e0 = exp2_approx(fmaf(s[n][t][2 * r], qs[n][0], -z0));
            const float e1 = exp2_approx(fmaf(s[n][t][2 * r + 1], qs[n][1], -z1));
            l[n][0] += e0;
            l[n][1] += e1;
            pk[t][r] = pack_f16x2(e0, e1);
          }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) pt[n][t][r] = movmatrix_trans(pk[t][r]);
      }

      // ---- output
      const uint32_t va = st + S::kV + lane * S::kPitch;
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        uint32_t pb[NB][2][2];
        uint4 f = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!kNv) f = lds128(st + S::kScaleV + i * 64 + c * 16);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          pb[n][0][0] = kNv ? pt[n][0][0] : hmul2(pt[n][0][0], f.x);
          pb[n][0][1] = kNv ? pt[n][0][1] : hmul2(pt[n][0][1], f.y);
          pb[n][1][0] = kNv ? pt[n][1][0] : hmul2(pt[n][1][0], f.z);
          pb[n][1][1] = kNv ? pt[n][1][1] : hmul2(pt[n][1][1], f.w);
        }
        uint32_t v[4];
        ldmatrix4_trans(v, va + i * 16);
        uint32_t h[4][4];  // [8 positions][code]: that code of positions 2c and 2c + 1
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t e[4];
          decode_word(v[k], e);  // codes 0, 1 | 2, 3 of position 2c, then of 2c + 1
          h[k][0] = __byte_perm(e[0], e[2], 0x5410);
          h[k][1] = __byte_perm(e[0], e[2], 0x7632);
          h[k][2] = __byte_perm(e[1], e[3], 0x5410);
          h[k][3] = __byte_perm(e[1], e[3], 0x7632);
          if constexpr (kNv) {
            const uint32_t f =
                e4m3x2_to_f16x2(lds16(st + S::kScaleV + (2 * i + (g >> 2)) * kStep + 8 * k + 2 * c));
#pragma unroll
            for (int n = 0; n < 4; ++n) h[k][n] = hmul2(h[k][n], f);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            mma16816(o[n][i][0], h[2 * t][0], h[2 * t][1], h[2 * t + 1][0], h[2 * t + 1][1], pb[n][t][0], pb[n][t][1]);
            mma16816(o[n][i][1], h[2 * t][2], h[2 * t][3], h[2 * t + 1][2], h[2 * t + 1][3], pb[n][t][0], pb[n][t][1]);
          }
      }
    }
    cp_wait<0>();
    const bool in_ring = kCluster || joined;
    if (in_ring) __syncwarp();  // the ring takes the part

    // ---- the result, or this part of it
#pragma unroll
    for (int k = 4; k < 32; k *= 2)
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) l[j >> 1][j & 1] += __shfl_xor_sync(0xFFFFFFFFu, l[j >> 1][j & 1], k);
    // slot unit + warp: the shares are consecutive, so no two parts have the same
    const int64_t unit_slot = static_cast<int64_t>(b) * units_per_seq + unit;
    auto store_part = [&](int holder, int h, int quad, float4 v) {
      float* to = p.part_o + ((unit_slot + holder) * kHeads + h) * D + quad * 4;
      if (MXFP4_IN_BOUNDS(p, kDbgPart, to, 16)) *reinterpret_cast<float4*>(to) = v;
    };
    auto store_part_sum = [&](int holder, int h, float top, float sum) {
      float* to = p.part_ml + ((unit_slot + holder) * kHeads + h) * 2;
      if (MXFP4_IN_BOUNDS(p, kDbgPart, to, 8)) *reinterpret_cast<float2*>(to) = make_float2(top, sum);
    };
    const int64_t head_at = static_cast<int64_t>(b) * p.num_q_heads + head0;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {  // heads 2c and 2c + 1; four values of each 32 in a lane
      const int n = j >> 1, e = j & 1, h = n * kColumns + 2 * c + e;
      const float top = m[n][e], sum = l[n][e] * kLower;
      if (h >= heads) continue;
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        // MXFP4: 2^(vref - 127); a block that met the NaN scale is NaN
        float f = kLower;
        if constexpr (!kNv)
          f = vref[i] == 255 ? __uint_as_float(0x7FC00000u) : scale_from_e8m0(vref[i]) * kLower;
        const float4 v = make_float4(o[n][i][0][e] * f, o[n][i][0][2 + e] * f, o[n][i][1][e] * f, o[n][i][1][2 + e] * f);
        const int d = i * 32 + 4 * g;
        if (in_ring) {
          sts128(ring + (h * D + d) * 4, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                 __float_as_uint(v.w));
        } else if (!whole) {
          store_part(worker, h, i * 8 + g, v);
        } else {
          store_out<kNv>(p, head_at + h, d, D, v, sum);
        }
      }
      if (g == 0) {
        if (in_ring) {
          sts64(ring + (kHeads * D + h * 2) * 4, __float_as_uint(top), __float_as_uint(sum));
        } else if (!whole) {
          store_part_sum(worker, h, top, sum);
        } else {
          store_lse(p, head_at + h, sum, top);
        }
      }
    }
    if constexpr (kCluster) {
      __syncwarp();
      cluster_sync();
      join_rings<DB, true, kHeads>(smem_u32(smem), kStages * S::kBytes, ctas, heads,
                           [&](int h, int quad, float4 v, float sum, float top) {
                             store_out<kNv>(p, head_at + h, 4 * quad, D, v, sum);
                             if (quad == 0) store_lse(p, head_at + h, sum, top);
                           });
      __syncwarp();
      cluster_sync();  // no CTA leaves while its parts are read
    } else if (joined) {  // this warp's last unit: the barrier is the CTA's
      __syncthreads();
      join_rings<DB, false, kHeads>(smem_u32(smem), kStages * S::kBytes, 1, heads,
                            [&](int h, int quad, float4 v, float sum, float top) {
                              if (whole) {
                                store_out<kNv>(p, head_at + h, 4 * quad, D, v, sum);
                                if (quad == 0) store_lse(p, head_at + h, sum, top);
                              } else {
                                store_part(worker - warp, h, quad, v);
                                if (quad == 0) store_part_sum(worker - warp, h, top, sum);
                              }
                            });
    }
  }
  if (!kCluster && p.workers > 0 && lane == 0 && MXFP4_IN_BOUNDS(p, kDbgPart, p.bad + worker, 4)) p.bad[worker] = bad;
  pdl_release();
}

__global__ void __launch_bounds__(kThreads) attention_status_kernel(const AttentionParams p) {
  pdl_wait();
  pdl_release();
  write_status(p);
}

// Joins the parts of each head, and writes what an empty sequence gives.  Four
// values of the output to a lane; with few parts to a head a warp takes them
// all (kPerHead 1), with many a CTA of 16 warps shares them.
template <bool kNv, int kPerHead>
__global__ void __launch_bounds__(kPerHead == 1 ? kThreads : 32 * kPerHead)
    attention_join_kernel(const AttentionParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int word = p.status != nullptr;
  if (word && blockIdx.x == 0) {
    // status word: what the warps met, and every length
    int bad = 0, lo, hi;
#pragma unroll 8
    for (int w = threadIdx.x; w < p.workers; w += blockDim.x)
      if (MXFP4_IN_BOUNDS(p, kDbgPart, p.bad + w, 4)) bad |= p.bad[w];
    for (int64_t b = threadIdx.x; b < p.num_seqs; b += blockDim.x) bad |= !positions(p, static_cast<int>(b), lo, hi);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && MXFP4_IN_BOUNDS(p.more, kDbgStatus, p.status, 4)) *p.status = bad ? -7 : 0;
    return;
  }
  const int64_t head = kPerHead == 1 ? static_cast<int64_t>(blockIdx.x - word) * kWarps + warp : blockIdx.x - word;
  if (head >= static_cast<int64_t>(p.num_seqs) * p.num_q_heads) return;
  const int b = static_cast<int>(head / p.num_q_heads), h = static_cast<int>(head - static_cast<int64_t>(b) * p.num_q_heads);
  const int kvh = h / p.group, in_group = h - kvh * p.group;
  const int64_t unit = (static_cast<int64_t>(b) * p.chunks + in_group / p.columns) * p.num_kv_heads + kvh;
  const int quads = p.head_dim / 4;
  float top = -INFINITY, sum = 0.0f;
  float4 acc[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (steps_of(p, b) > 0) {
    if (!MXFP4_IN_BOUNDS(p, kDbgPart, p.parts + unit, 16)) return;
    const int4 who = p.parts[unit];
    const Parts parts{who.x, who.y, who.z, who.w};
    const int n = parts.count();
    if (n == 1) return;  // written already
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + in_group % p.columns;
    const float4* po = reinterpret_cast<const float4*>(p.part_o) + in_group % p.columns * quads;
    // one pass, kBatch parts' loads in flight
    constexpr int kBatch = 6;
    for (int s0 = kPerHead == 1 ? 0 : warp; s0 < n; s0 += kBatch * kPerHead) {
      float2 part[kBatch];
      float4 v[kBatch][2];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int s = s0 + k * kPerHead;
        const int64_t slot = (unit + parts.warp(s)) * p.columns;
        part[k] = s < n && MXFP4_IN_BOUNDS(p, kDbgPart, ml + slot, 8) ? ml[slot] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[k][i] = s < n && i * 32 + lane < quads &&
                            MXFP4_IN_BOUNDS(p, kDbgPart, po + (slot * quads + i * 32 + lane), 16)
                        ? po[slot * quads + i * 32 + lane]
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float x = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) x = fmaxf(x, part[k].x);
      const float z = x == -INFINITY ? 0.0f : x;
      const float keep = exp2_approx(top - z);
      top = x;
      sum *= keep;
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i] = make_float4(acc[i].x * keep, acc[i].y * keep, acc[i].z * keep, acc[i].w * keep);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = exp2_approx(part[k].x - z);
        sum += part[k].y * f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[i].x += v[k][i].x * f;
          acc[i].y += v[k][i].y * f;
          acc[i].z += v[k][i].z * f;
          acc[i].w += v[k][i].w * f;
        }
      }
    }
  }
  if constexpr (kPerHead == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i * 32 + lane < quads) store_out<kNv>(p, head, 4 * (i * 32 + lane), p.head_dim, acc[i], sum);
    if (lane == 0) store_lse(p, head, sum, top);
  } else {
    __shared__ float4 s_acc[kPerHead][64];
    __shared__ float s_sum[kPerHead], s_top[kPerHead];
#pragma unroll
    for (int i = 0; i < 2; ++i) s_acc[warp][i * 32 + lane] = acc[i];
    if (lane == 0) {
      s_sum[warp] = sum;
      s_top[warp] = top;
    }
    __syncthreads();
    if (threadIdx.x < quads) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float l = 0.0f, x = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPerHead; ++w) x = fmaxf(x, s_top[w]);
      const float z = x == -INFINITY ? 0.0f : x;
#pragma unroll
      for (int w = 0; w < kPerHead; ++w) {
        const float4 v = s_acc[w][threadIdx.x];
        const float f = exp2_approx(s_top[w] - z);
        a.x += v.x * f;
        a.y += v.y * f;
        a.z += v.z * f;
        a.w += v.w * f;
        l += s_sum[w] * f;
      }
      store_out<kNv>(p, head, 4 * threadIdx.x, p.head_dim, a, l);
      if (threadIdx.x == 0) store_lse(p, head, l, x);
    }
  }
  // Not before the end: the next call's warps have even shares, so its CTAs
  // should find the SMs free of this kernel's.
  pdl_release();
}

template <bool kNv, int DB, int NB>
cudaError_t launch_dim(const AttentionParams& p, unsigned grid, cudaStream_t stream) {
  using S = Stage<kNv, DB>;
  static std::atomic<uint64_t> ready[2] = {};
  const bool cluster = p.ctas > 0;
  const auto kernel = cluster ? attention_kernel<kNv, DB, true, NB> : attention_kernel<kNv, DB, false, NB>;
  const int smem = kWarps * stages_of(DB, cluster) * S::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem, ready[cluster]); e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, grid, kThreads, smem, stream, p.ctas, p);
}
template <bool kNv, int DB>
cudaError_t launch_columns(const AttentionParams& p, unsigned grid, cudaStream_t stream) {
  return p.columns == kColumns ? launch_dim<kNv, DB, 1>(p, grid, stream) : launch_dim<kNv, DB, 2>(p, grid, stream);
}

template <bool kNv>
cudaError_t launch_format(const AttentionParams& p, unsigned grid, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  switch (p.head_dim / 32) {
    case 1: e = launch_columns<kNv, 1>(p, grid, stream); break;
    case 2: e = launch_columns<kNv, 2>(p, grid, stream); break;
    case 3: e = launch_columns<kNv, 3>(p, grid, stream); break;
    case 4: e = launch_columns<kNv, 4>(p, grid, stream); break;
    case 5: e = launch_dim<kNv, 5, 1>(p, grid, stream); break;
    case 6: e = launch_dim<kNv, 6, 1>(p, grid, stream); break;
    case 7: e = launch_dim<kNv, 7, 1>(p, grid, stream); break;
    default: e = launch_dim<kNv, 8, 1>(p, grid, stream); break;
  }
  if (e != cudaSuccess || p.workers == 0) return e;
  const int64_t heads = static_cast<int64_t>(p.num_seqs) * p.num_q_heads;
  const int64_t units = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * p.chunks;
  const unsigned word = p.status != nullptr;
  // 1, 4 or 16 warps to a head.  One sequence of 131072 (head_dim 64, 304 warps to a
  // unit): 37.4, 29.8 and 28.1 us; 64 sequences of 8192 (4): 99, 105 and 145; 4 of
  // 32768 (head_dim 256, 152): 36.3, 33.2 and 33.2.
  if (p.workers >= 32 * units)
    return launch_pdl(attention_join_kernel<kNv, 16>, static_cast<unsigned>(heads) + word, 32 * 16, 0, stream, p);
  if (p.workers >= 6 * units)
    return launch_pdl(attention_join_kernel<kNv, 4>, static_cast<unsigned>(heads) + word, 32 * 4, 0, stream, p);
  return launch_pdl(attention_join_kernel<kNv, 1>, static_cast<unsigned>((heads + kWarps - 1) / kWarps) + word,
                    kThreads, 0, stream, p);
}

// CTAs that `sms` SMs, the current device's, hold at once.
int64_t resident_ctas(int sms, int32_t head_dim, bool cluster, int columns) {
  return static_cast<int64_t>(sms) * ctas_of(head_dim / 32, cluster, columns / kColumns);
}
// Contexts that one warp takes whole: a step.
bool one_step(int64_t max_len) { return max_len <= kStep; }
// CTAs of the cluster that takes a unit, as many as have a step for each warp and
// are resident together, where that leaves a warp kFewSteps steps at most; else 0.
// Without the second kernel and the workspace, but with the SMs idle that the
// clusters leave: 8.5 -> 6.5 us for one sequence of 700 positions (64 heads on 8,
// head_dim 128), 26.9 -> 21.8 for 64 of up to 1024 (8 steps); at 12 steps, one
// of 12000, 14.3 -> 15.8.
int cluster_ctas(int sms, int64_t units, int32_t head_dim, int columns, int64_t max_len) {
  constexpr int64_t kFewSteps = 8;
  constexpr int kMost = 8;  // the portable size
  if (one_step(max_len)) return 0;
  const int64_t steps = (max_len + kStep - 1) / kStep, most = resident_ctas(sms, head_dim, true, columns);
  int ctas = 1;
  while (ctas < kMost && steps > ctas * kWarps && units * ctas * 2 <= most) ctas *= 2;
  return units * ctas <= most && steps <= kFewSteps * ctas * kWarps ? ctas : 0;
}

// Warps that share the positions of all sequences: as many as the GPU holds at
// once, so that all end together; 0 for contexts so short that a warp or a
// cluster takes a unit whole.
int shared_workers(int sms, int64_t units, int32_t head_dim, int columns, int64_t max_len) {
  if (one_step(max_len) || cluster_ctas(sms, units, head_dim, columns, max_len) > 0) return 0;
  const int64_t resident = resident_ctas(sms, head_dim, false, columns) * kWarps;
  const int64_t most = (units * ((max_len + kStep - 1) / kStep) + kWarps - 1) / kWarps * kWarps;
  return static_cast<int>(most < resident ? most : resident);
}

// Query heads of a unit: two column blocks, for which the cache is decoded once,
// where a kv head has more than 8, the registers hold them, and each warp has 2.5
// steps or more with one.  128 heads on 8 of 128: 32 sequences of up to 4096 55.3 ->
// 48.9 us; one of 700, with half as many warps to share it, 7.6 -> 8.7.  64 heads on
// 4 of 64, 8 of 4096 (2.7 steps): 13.0 -> 10.4; 80 on 5 of 128, 16 of 1000 (2.1):
// 11.2 -> 11.9.
int columns_of(int sms, int64_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
               int64_t max_len) {
  const int group = num_q_heads / num_kv_heads;
  if (group <= kColumns || head_dim > 128) return kColumns;
  const int64_t units = num_seqs * num_kv_heads * ((group + kColumns - 1) / kColumns);
  const int64_t steps = units * ((max_len + kStep - 1) / kStep);
  return 2 * steps >= 5 * kWarps * resident_ctas(sms, head_dim, true, kColumns) ? 2 * kColumns : kColumns;
}

}  // namespace

int64_t attention_workspace_floats(int64_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int64_t max_len) {
  if (num_seqs == 0 || num_q_heads == 0 || head_dim == 0) return 0;
  const int sms = sm_count(), group = num_q_heads / num_kv_heads;
  const int columns = columns_of(sms, num_seqs, num_q_heads, num_kv_heads, head_dim, max_len);
  const int64_t units = num_seqs * num_kv_heads * ((group + columns - 1) / columns);
  const int workers = shared_workers(sms, units, head_dim, columns, max_len);
  return workers > 0 ? (units + workers) * columns * (head_dim + 2) + 4 * units + workers : 0;
}

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
  // without pages every position is out of range
  p.max_len = c.num_pages > 0 ? a.max_pages * c.page_size : 0;
  p.num_seqs = static_cast<int32_t>(a.num_seqs);
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = c.num_heads;
  p.num_pages = static_cast<int32_t>(c.num_pages);
  p.page_size = c.page_size;
  p.head_dim = c.head_dim;
  p.window = a.window;
  p.scale_bytes = static_cast<uint64_t>(c.num_pages) * c.page_size * c.num_heads * (c.head_dim / (c.nvfp4 ? 16 : 32));
  p.f16 = c.f16;
  p.softmax_scale = a.softmax_scale;
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.more.dbg, kDbgLens, a.seq_lens, a.num_seqs * 4);
  debug_range(p.more.dbg, kDbgStatus, a.status, a.status ? 4 : 0);
  debug_range(p.dbg, kDbgTable, a.page_table,
              a.num_seqs > 0 ? ((a.num_seqs - 1) * a.table_stride + a.max_pages) * 4 : 0);
#endif
  if (a.num_q_heads == 0 || c.head_dim == 0) {  // the status word alone
    if (a.status == nullptr) return cudaSuccess;
    return launch_pdl(attention_status_kernel, 1, kThreads, 0, stream, p);
  }
  p.group = a.num_q_heads / c.num_heads;
  const int sms = sm_count();
  p.columns = columns_of(sms, a.num_seqs, a.num_q_heads, c.num_heads, c.head_dim, a.max_pages * c.page_size);
  p.chunks = (p.group + p.columns - 1) / p.columns;
  const int64_t units = a.num_seqs * c.num_heads * p.chunks;
  p.workers = shared_workers(sms, units, c.head_dim, p.columns, a.max_pages * c.page_size);
  p.ctas = cluster_ctas(sms, units, c.head_dim, p.columns, a.max_pages * c.page_size);
  p.part_o = a.workspace;
  p.part_ml = p.part_o + (units + p.workers) * p.columns * c.head_dim;
  p.parts = reinterpret_cast<int4*>(p.part_ml + (units + p.workers) * p.columns * 2);
  p.bad = reinterpret_cast<int32_t*>(p.parts + units);
#ifdef MXFP4_DEBUG_BOUNDS
  const int64_t rows = c.num_pages * c.page_size * c.num_heads;
  debug_range(p.dbg, kDbgQ, a.q, a.num_seqs > 0
      ? ((a.num_seqs - 1) * a.q_seq_stride + (a.num_q_heads - 1) * a.q_head_stride + c.head_dim) * 2 : 0);
  for (int i = 0; i < 2; ++i) {
    debug_range(p.dbg, kDbgCodes0 + i, c.codes[i], rows * (c.head_dim / 2));
    debug_range(p.dbg, kDbgScales0 + i, c.scales[i], rows * (c.head_dim / (c.nvfp4 ? 16 : 32)));
  }
  debug_range(p.more.dbg, kDbgLse, a.lse, a.lse ? a.num_seqs * a.num_q_heads * 4 : 0);
  debug_range(p.dbg, kDbgOut, a.out, a.num_seqs * a.num_q_heads * c.head_dim * 2);
  debug_range(p.dbg, kDbgPart, a.workspace,
              p.workers > 0 ? ((units + p.workers) * p.columns * (c.head_dim + 2) + 4 * units + p.workers) * 4 : 0);
#endif
  const int64_t word = a.status != nullptr;
  const int64_t grid = p.workers > 0 ? p.workers / kWarps
                       : p.ctas > 0  ? (units + word) * p.ctas
                                     : (units + kWarps - 1) / kWarps + word;
  if (grid == 0) return cudaSuccess;
  return c.nvfp4 ? launch_format<true>(p, static_cast<unsigned>(grid), stream)
                 : launch_format<false>(p, static_cast<unsigned>(grid), stream);
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

// topk.cu — the router's choice for sm_103a: the top_k experts of every token
// and their weights (formulas in include/mxfp4.h).
//
// A warp to a token; each lane holds the picks of some experts (-infinity: out), and
// a round of the choice is one redux.max over the lanes' best picks and one redux.min
// over the indices that have it: equal picks go to the lowest index.  A lane knows its two best, and looks
// through its picks again when both are taken.
//
// Without a bias and group sums the picks are the logits, and exact.  Else they
// are float32 scores plus bias, and two closer than their errors may be in the
// wrong order.  The rounds go on while a pick is that near the last chosen, and
// where any two neighbours are near each other (about one token in 500 with 384
// experts of ordinary spread) the ones found, one to a lane, are computed in 64
// bits and ranked again.  Groups near the last that stays are compared in 64 bits
// as well.  Where more than 32 picks are near one another, choose_exactly finds
// them one by one.
//
// Instructions bound it: 16384 tokens on 384 experts take 16 us by their logits, 20 with
// sigmoid and bias, 26 to 30 in 8 groups by their two best (1330 instructions to a token;
// the bytes alone would be 4 us), of which the ranking in 64 bits 3 and 7.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxfp4_device.cuh"
#include "mxfp4_internal.h"
#include "../../include/mxfp4.h"

namespace mxfp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxPerLane = 32;  // keys in registers; more lie in shared memory
constexpr int kNear = 32;        // picks that are ranked at once, one to a lane

// A warp's words of shared memory: the picks (`held`: groups or kPer == 0), a bit for
// each expert, and those ranked; whole 16-byte pieces, as the picks are stored.
__host__ __device__ constexpr int warp_words(int E, bool held) {
  const int padded = (E + 31) / 32 * 32;
  return ((held ? padded : 0) + padded / 32 + kNear + 3) / 4 * 4;
}

struct TopkParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t ld;
  int32_t tokens;
  int32_t E;
  int32_t groups;
  int32_t size;  // experts of a group
  float inv_size;
  int32_t top_groups;
  int32_t top_k;
  float scale;
  bool sigmoid;
  bool group_sum2;
  bool renormalize;
  bool scored;   // keys are scores (plus bias), not logits
#ifdef MXFP4_DEBUG_BOUNDS
  DebugRanges dbg;
#endif
};

enum : int { kDbgLogits = 0, kDbgBias, kDbgIds, kDbgWeights };

template <LogitType kType>
__device__ __forceinline__ float logit_at(const TopkParams& p, int64_t row, int e) {
  if constexpr (kType == LogitType::kF32) {
    const float* at = static_cast<const float*>(p.logits) + row * p.ld + e;
    return MXFP4_IN_BOUNDS(p, kDbgLogits, at, 4) ? __ldg(at) : 0.0f;
  } else {
    const uint16_t* at = static_cast<const uint16_t*>(p.logits) + row * p.ld + e;
    const uint16_t v = MXFP4_IN_BOUNDS(p, kDbgLogits, at, 2) ? __ldg(at) : 0;
    if constexpr (kType == LogitType::kF16) return __half2float(__ushort_as_half(v));
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
}
__device__ __forceinline__ float bias_at(const TopkParams& p, int e) {
  if (p.bias == nullptr) return 0.0f;
  return MXFP4_IN_BOUNDS(p, kDbgBias, p.bias + e, 4) ? __ldg(p.bias + e) : 0.0f;
}

// e / size: (e + 1/2) / size is at least 1 / (2 size) >= 2^-14 from the next whole
// number (sizes are up to 8192), the product off by less than 2^-16 (it is under 32).
__device__ __forceinline__ int group_of(const TopkParams& p, int e) {
  return static_cast<int>((e + 0.5f) * p.inv_size);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// (volatile: all lanes take part, also where a branch behind it uses the result)
__device__ __forceinline__ float warp_most(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_least(float x) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kOut = -INFINITY;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// A pick in float32.  sigmoid: 1 / (1 + e^-l); softmax: e^(l - top) / sum.  With
// the fast exponential and division a score s is off by 2^-21 at most: s (1 - s)
// (2^-22 + |l| 2^-24) <= 2^-23 for e^-l, 2^-24 and 2^-23 for the addition and
// the division.  A softmax's sum of E terms, added by lanes and then in a tree,
// adds (E / 32 + 5) 2^-24.  The addition of the bias is off by 2^-24 of the pick.
__device__ __forceinline__ float pick32(const TopkParams& p, float l, float b, float top,
                                        float inv_sum) {
  if (!p.sigmoid) return fmaf(__expf(l - top), inv_sum, b);
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s + b;
}
// Twice what two neighbours of at most `m` may be off by together.
__device__ __forceinline__ float tolerance(const TopkParams& p, float m) {
  return (p.sigmoid ? 0x1p-20f : 0x1p-18f + 0x1p-27f * p.E) + 0x1p-21f * fabsf(m);
}

// The lanes' picks, in registers or (kPer == 0) in shared memory.
template <int kPer>
struct Picks {
  float v[kPer];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(int i, float k) { v[i] = k; }
  __device__ __forceinline__ int count() const { return kPer; }
};
template <>
struct Picks<0> {
  float* v;
  int n;
  __device__ __forceinline__ float get(int i) const { return v[i * 32]; }
  __device__ __forceinline__ void set(int i, float k) { v[i * 32] = k; }
  __device__ __forceinline__ int count() const { return n; }
};

// ---------------------------------------------------- the exact choice
struct Exact {
  int64_t row;
  float top;        // the largest logit, and in float32 and 64 bits the softmax's
  float inv_sum;    // sum's inverse
  double inv_sum64;
  uint32_t kept;    // groups that stay
  uint32_t* gone;   // a bit for each expert that has been taken
};

// e^x in 64 bits, to about 2^-52: x = n ln 2 + r with |r| <= ln(2) / 2 (Cody and Waite's
// reduction: ln 2 in two parts, the first its leading 40 bits, so that n times it is
// exact) and r's Taylor series to r^13 (r^14 / 14! < 2^-57), without a function call and
// its saved registers.  0 below -708, where a score no longer counts beside any other.
__device__ __forceinline__ double exp64(double x) {
  if (!(x > -708.0)) return 0.0;
  x = fmin(x, 709.0);
  const double n = rint(x * 1.4426950408889634);
  double r = fma(n, -0x1.62e42fefa2p-1, x);    // floor(2^40 ln 2) / 2^40
  r = fma(n, -0x1.9ef35793c7673p-41, r);       // and the rest
  double s = 1.0 / 6227020800.0;
  constexpr double kInverse[13] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                                   1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
#pragma unroll
  for (int i = 12; i >= 0; --i) s = fma(s, r, kInverse[i]);
  return s * __hiloint2double((static_cast<int>(n) + 1023) << 20, 0);
}
// 1 / x for 1 <= x <= 2^1023, by Newton's steps from a power of two's inverse and
// the float32 inverse of the rest.
__device__ __forceinline__ double inverse64(double x) {
  const int e = (__double2hiint(x) >> 20) - 1023;                   // x = m 2^e, 1 <= m < 2
  const double m = x * __hiloint2double((1023 - min(e, 1022)) << 20, 0);
  double y = __fdividef(1.0f, static_cast<float>(m));
#pragma unroll
  for (int i = 0; i < 3; ++i) y = fma(y, fma(-m, y, 1.0), y);
  return y * __hiloint2double((1023 - min(e, 1022)) << 20, 0);
}
__device__ __forceinline__ double pick64(const TopkParams& p, const Exact& x, float l, float b) {
  const double s = p.sigmoid ? inverse64(1.0 + exp64(-static_cast<double>(l)))
                             : exp64(static_cast<double>(l) - x.top) * x.inv_sum64;
  return s + b;
}

// The best of experts [lo, hi) that are not taken, of groups that stay; -1 if
// there is none.  All lanes call it and get the same.
template <LogitType kType>
__device__ int best_exactly(const TopkParams& p, const Exact& x, int lo, int hi, double& value) {
  const int lane = threadIdx.x & 31;
  const auto pick_at = [&](int e, float& l, float& b, float& v) {
    l = logit_at<kType>(p, x.row, e);
    b = bias_at(p, e);
    v = pick32(p, l, b, x.top, x.inv_sum);
    return finite(l) && finite(b) && !((x.gone[e >> 5] >> (e & 31)) & 1u) &&
           ((x.kept >> group_of(p, e)) & 1u);
  };
  float most = kOut;
  for (int e = lo + lane; e < hi; e += 32) {
    float l, b, v;
    if (pick_at(e, l, b, v)) most = fmaxf(most, v);
  }
  most = warp_most(most);
  if (most == kOut) return -1;
  const float from = most - tolerance(p, most);
  int at = INT32_MAX;
  double best = 0.0;
  float at_l = 0.0f, at_b = 0.0f;
  for (int e = lo + lane; e < hi; e += 32) {
    float l, b, v;
    if (!pick_at(e, l, b, v) || v < from) continue;
    if (at != INT32_MAX && l == at_l && b == at_b) continue;  // the same pick, further on
    const double d = pick64(p, x, l, b);
    if (at == INT32_MAX || d > best) best = d, at = e, at_l = l, at_b = b;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const double other = __shfl_xor_sync(kAll, best, d);
    const int from_e = __shfl_xor_sync(kAll, at, d);
    if (from_e != INT32_MAX &&
        (at == INT32_MAX || other > best || (other == best && from_e < at)))
      best = other, at = from_e;
  }
  value = best;
  return at;
}

template <LogitType kType>
__device__ __forceinline__ double softmax_inverse(const TopkParams& p, int64_t row, float top) {
  double sum = 0.0;
  for (int e = threadIdx.x & 31; e < p.E; e += 32) {
    const float l = logit_at<kType>(p, row, e);
    if (finite(l)) sum += exp64(static_cast<double>(l) - top);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  return inverse64(sum);
}

__device__ __forceinline__ void none_gone(const TopkParams& p, uint32_t* gone) {
  __syncwarp();
  for (int i = threadIdx.x & 31; i < (p.E + 31) / 32; i += 32) gone[i] = 0;
  __syncwarp();
}
__device__ __forceinline__ void take(uint32_t* gone, int e) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) gone[e >> 5] |= 1u << (e & 31);
  __syncwarp();
}

// Of the groups in `near`, the `count` best by their values in 64 bits: of those
// of a group's `held` picks that may be its best (or two best) in exact terms.
// Lane g: group g's best pick, or with group sums its second (kOut: it has one).
template <LogitType kType>
__device__ __forceinline__ uint32_t best_groups_exactly(const TopkParams& p, Exact x, const float* held, float lowest,
                                                     uint32_t near, int count) {
  const int lane = threadIdx.x & 31;
  if (!p.sigmoid) x.inv_sum64 = softmax_inverse<kType>(p, x.row, x.top);
  constexpr double kNone = -1.7976931348623157e308;
  double mine = kNone;
  bool open = false;
  for (uint32_t rest = near; rest != 0; rest &= rest - 1) {
    const int g = __ffs(rest) - 1;
    const float low = __shfl_sync(kAll, lowest, g);
    const float from = low != kOut ? low - tolerance(p, low) : kOut;
    double first = kNone, second = kNone;
    for (int i = lane; i < p.size; i += 32) {
      const int e = g * p.size + i;
      const float v = held[e];
      if (v == kOut || v < from) continue;
      const double d = pick64(p, x, logit_at<kType>(p, x.row, e), bias_at(p, e));
      second = fmax(second, fmin(first, d));
      first = fmax(first, d);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double a = __shfl_xor_sync(kAll, first, d), b = __shfl_xor_sync(kAll, second, d);
      second = fmax(fmin(first, a), fmax(second, b));
      first = fmax(first, a);
    }
    if (lane == g) {
      open = first != kNone;
      mine = p.group_sum2 && second != kNone ? first + second : first;
    }
  }
  uint32_t kept = 0;
  for (int j = 0; j < count; ++j) {
    double best = mine;
    int at = open ? lane : INT32_MAX;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double other = __shfl_xor_sync(kAll, best, d);
      const int from = __shfl_xor_sync(kAll, at, d);
      if (from != INT32_MAX && (at == INT32_MAX || other > best || (other == best && from < at)))
        best = other, at = from;
    }
    if (at == INT32_MAX) break;
    kept |= 1u << at;
    if (lane == at) open = false;
  }
  return kept;
}

// Lane j's chosen expert (-1: none), found one by one in 64 bits.
template <LogitType kType>
__device__ __forceinline__ int choose_exactly(const TopkParams& p, const Exact& x) {
  none_gone(p, x.gone);
  int id = -1;
  double value;
  for (int j = 0; j < p.top_k; ++j) {
    const int e = best_exactly<kType>(p, x, 0, p.E, value);
    if (e < 0) break;
    if (static_cast<int>(threadIdx.x & 31) == j) id = e;
    take(x.gone, e);
  }
  return id;
}

// The lanes' experts (-1: none) ranked by their picks in 64 bits: lane j gets the
// j-th.  `order`: 32 words of the warp's.
template <LogitType kType>
__device__ __forceinline__ int rank_exactly(const TopkParams& p, const Exact& x, int id, int found, uint32_t* order) {
  const int lane = threadIdx.x & 31;
  double mine = 0.0;
  if (id >= 0) mine = pick64(p, x, logit_at<kType>(p, x.row, id), bias_at(p, id));
  int rank = 0;
  for (int j = 0; j < found; ++j) {
    const double other = __shfl_sync(kAll, mine, j);
    const int e = __shfl_sync(kAll, id, j);
    rank += other > mine || (other == mine && e < id);
  }
  __syncwarp();
  if (id >= 0) order[rank] = id;
  __syncwarp();
  return lane < found ? static_cast<int>(order[lane]) : -1;
}

// What the rounds found near one another (`many`: more than kNear), in exact order.
template <LogitType kType>
__device__ __forceinline__ int order_exactly(const TopkParams& p, Exact x, int id, int found, bool many, uint32_t* order) {
  if (!p.sigmoid) x.inv_sum64 = softmax_inverse<kType>(p, x.row, x.top);
  return many ? choose_exactly<kType>(p, x) : rank_exactly<kType>(p, x, id, found, order);
}

// ------------------------------------------------------------ the kernel
// A lane's key i is that of expert expert_of(i): with kVec == 4 four consecutive
// experts in a load, else one.
template <int kVec>
__device__ __forceinline__ int key_part(int i) {
  return kVec == 4 ? (i >> 2) * 128 + (i & 3) : i * 32;
}
template <int kVec>
__device__ __forceinline__ int expert_of(int i) {
  return key_part<kVec>(i) + static_cast<int>(threadIdx.x & 31) * kVec;
}
// The logits (infinity: no expert) or biases of keys i to i + kVec - 1.
template <int kVec, LogitType kType>
__device__ __forceinline__ void load_logits(const TopkParams& p, int64_t row, int i, float (&l)[kVec]) {
  const int e = expert_of<kVec>(i);
#pragma unroll
  for (int j = 0; j < kVec; ++j) l[j] = INFINITY;
  if (e >= p.E) return;
  if constexpr (kVec == 1) {
    l[0] = logit_at<kType>(p, row, e);
  } else if constexpr (kType == LogitType::kF32) {
    const float* at = static_cast<const float*>(p.logits) + row * p.ld + e;
    if (!MXFP4_IN_BOUNDS(p, kDbgLogits, at, 16)) return;
    const float4 v = __ldg(reinterpret_cast<const float4*>(at));
    l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
  } else {
    const uint16_t* at = static_cast<const uint16_t*>(p.logits) + row * p.ld + e;
    if (!MXFP4_IN_BOUNDS(p, kDbgLogits, at, 8)) return;
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
    if constexpr (kType == LogitType::kF16) {
      l[0] = half_lo_to_f32(v.x), l[1] = half_hi_to_f32(v.x), l[2] = half_lo_to_f32(v.y), l[3] = half_hi_to_f32(v.y);
    } else {
      l[0] = __uint_as_float(v.x << 16), l[1] = __uint_as_float(v.x & 0xFFFF0000u);
      l[2] = __uint_as_float(v.y << 16), l[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  }
}
template <int kVec>
__device__ __forceinline__ void load_biases(const TopkParams& p, int i, float (&b)[kVec]) {
  const int e = expert_of<kVec>(i);
#pragma unroll
  for (int j = 0; j < kVec; ++j) b[j] = 0.0f;
  if (p.bias == nullptr || e >= p.E) return;
  if constexpr (kVec == 1) {
    b[0] = bias_at(p, e);
  } else if (MXFP4_IN_BOUNDS(p, kDbgBias, p.bias + e, 16)) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p.bias + e));
    b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
  }
}

template <int kPer, int kVec, LogitType kType>
__global__ void __launch_bounds__(kThreads, 1) moe_topk_kernel(const TopkParams p) {
  extern __shared__ __align__(16) float s_words[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int padded = (p.E + 31) / 32 * 32;
  const bool in_smem = kPer == 0 || p.groups > 1;
  float* held = s_words + warp * warp_words(p.E, in_smem);
  uint32_t* gone = reinterpret_cast<uint32_t*>(held + (in_smem ? padded : 0));
  uint32_t* order = gone + padded / 32;
  pdl_wait();
  pdl_release();
  if (row >= p.tokens) return;

  Picks<kPer> picks;
  if constexpr (kPer == 0) picks.v = held + lane, picks.n = padded / 32;
  float top = kOut, inv_sum = 1.0f;
  const bool direct = p.scored && p.sigmoid;  // a logit's pick needs no other's
#pragma unroll
  for (int i = 0; i < picks.count(); i += kVec) {
    float l[kVec], b[kVec];
    load_logits<kVec, kType>(p, row, i, l);
    if (direct) load_biases<kVec>(p, i, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float v = l[j];
      if (direct) v = pick32(p, v, b[j], 0.0f, 1.0f);
      v = finite(l[j]) && finite(v) ? v : kOut;
      picks.set(i + j, v);
      if (!p.sigmoid) top = fmaxf(top, v);
    }
  }
  if (!p.sigmoid) {
    top = warp_most(top);
    if (p.scored || !p.renormalize) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < picks.count(); ++i) {
        const float l = picks.get(i);
        if (l != kOut) sum += expf(l - top);
      }
      inv_sum = __fdividef(1.0f, warp_sum(sum));
    }
    if (p.scored) {
#pragma unroll
      for (int i = 0; i < picks.count(); i += kVec) {
        float b[kVec];
        load_biases<kVec>(p, i, b);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float l = picks.get(i + j), v = pick32(p, l, b[j], top, inv_sum);
          picks.set(i + j, l != kOut && finite(v) ? v : kOut);
        }
      }
    }
  }
  Exact x{row, top, inv_sum, 0.0, kAll, gone};  // the sum in 64 bits: where it is needed

  if (p.groups > 1) {
    if constexpr (kPer > 0) {
#pragma unroll
      for (int i = 0; i < kPer; i += kVec) {
        const int e = expert_of<kVec>(i);
        if constexpr (kVec == 4) {
          if (e < p.E) *reinterpret_cast<float4*>(held + e) = make_float4(picks.v[i], picks.v[i + 1], picks.v[i + 2], picks.v[i + 3]);
        } else {
          if (e < p.E) held[e] = picks.v[i];
        }
      }
    }
    __syncwarp();
    // 32 / share lanes to a group, its two best merged over them
    int share = 1;
    while (share < p.groups) share <<= 1;
    const int lanes = 32 / share;
    const int g = lane / lanes;
    float a = kOut, b = kOut;
    if (g < p.groups)
#pragma unroll 4
      for (int i = lane % lanes; i < p.size; i += lanes) {
        const float k = held[g * p.size + i];
        b = fmaxf(b, fminf(a, k));
        a = fmaxf(a, k);
      }
    for (int d = lanes >> 1; d > 0; d >>= 1) {
      const float oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    const float lowest = p.group_sum2 && b != kOut ? b : a;
    float size = a != kOut ? fabsf(a) : 0.0f;
    if (p.group_sum2 && b != kOut) size += fabsf(b), a += b;
    // a group to a lane: those before it are larger, or equal and of a lower index
    const float value = __shfl_sync(kAll, a, lane < p.groups ? lane * lanes : 0);
    const float mine = lane < p.groups ? value : kOut;
    int before = 0;
    for (int j = 0; j < p.groups; ++j) {
      const float other = __shfl_sync(kAll, mine, j);
      before += other > mine || (other == mine && j < lane);
    }
    const bool open = mine != kOut, in = open && before < p.top_groups;
    uint32_t kept = __ballot_sync(kAll, in);
    if (p.scored && p.top_groups < p.groups) {
      // what could be on either side of the border in exact terms
      const float tol = 2.0f * tolerance(p, warp_most(size));
      const float first_out = warp_most(open && !in ? mine : kOut), border = warp_least(in ? mine : INFINITY);
      if (first_out != kOut && border - first_out <= tol) {
        const uint32_t near = __ballot_sync(kAll, open && fabsf(mine - border) <= 2.0f * tol);
        const uint32_t sure = kept & ~near;
        const float low = __shfl_sync(kAll, lowest, lane < p.groups ? lane * lanes : 0);
        kept = sure | best_groups_exactly<kType>(p, x, held, low, near, p.top_groups - __popc(sure));
      }
    }
    x.kept = kept;
    // (read again: nothing is held over the calls above)
    if (kVec == 4 && kPer > 0 && (p.size & 3) == 0) {  // four experts of a load are of one group
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const int e = expert_of<kVec>(i);
        const bool in_kept = e < p.E && ((kept >> group_of(p, e)) & 1u);
        const float4 v = in_kept ? *reinterpret_cast<const float4*>(held + e) : make_float4(kOut, kOut, kOut, kOut);
        picks.set(i, v.x), picks.set(i + 1, v.y), picks.set(i + 2, v.z), picks.set(i + 3, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < picks.count(); ++i) {
        const int e = expert_of<kVec>(i);
        picks.set(i, e < p.E && ((kept >> group_of(p, e)) & 1u) ? held[e] : kOut);
      }
    }
  }

  // the rounds
  int id = -1, found = 0, best_i = 0, next_i = 0;
  float best = kOut, next = kOut;
  bool fresh = true;  // `next` is known
#pragma unroll
  for (int i = 0; i < picks.count(); ++i) {
    const float k = picks.get(i);
    const bool first = k > best, second = k > next;
    next = fminf(fmaxf(k, next), best);
    next_i = first ? best_i : second ? key_part<kVec>(i) : next_i;
    best = fmaxf(k, best);
    best_i = first ? key_part<kVec>(i) : best_i;
  }
  bool near = false, many = false;
  float last = 0.0f, kth = 0.0f;
  for (;;) {
    const float m = warp_most(best);
    if (m == kOut) break;
    if (found >= p.top_k) {
      if (kth - m > tolerance(p, kth)) break;
      if (found == kNear) {
        many = true;
        break;
      }
    }
    if (p.scored) {
      if (found > 0) near |= last - m <= tolerance(p, last);
      last = m;
    }
    const int mine = best == m ? best_i + lane * kVec : INT32_MAX;  // (best_i: key_part)
    const int e = __reduce_min_sync(kAll, mine);
    if (lane == found) id = e;
    if (++found == p.top_k) {
      kth = m;
      if (!p.scored) break;
    }
    if (mine == e) {
      if (fresh) {
        best = next, best_i = next_i, fresh = false;
      } else {
        // the two best behind the last taken in their order
        const float limit = best;
        const int limit_i = best_i;
        best = next = kOut;
#pragma unroll
        for (int i = 0; i < picks.count(); ++i) {
          float k = picks.get(i);
          k = k < limit || (k == limit && key_part<kVec>(i) > limit_i) ? k : kOut;
          const bool first = k > best, second = k > next;
          next = fminf(fmaxf(k, next), best);
          next_i = first ? best_i : second ? key_part<kVec>(i) : next_i;
          best = fmaxf(k, best);
          best_i = first ? key_part<kVec>(i) : best_i;
        }
        fresh = true;
      }
    }
  }
  if (p.scored && (near || many)) id = order_exactly<kType>(p, x, id, found, many, order);
  if (lane >= p.top_k) id = -1;

  // the weights, from the chosen logits (a renormalised softmax is the chosen
  // ones' own; small sigmoids are raised together, so that they do not vanish)
  float w = 0.0f;
  const float l = id >= 0 ? logit_at<kType>(p, row, id) : -INFINITY;
  float high = p.sigmoid ? 0.0f : top;
  if (p.renormalize) high = p.sigmoid ? fminf(warp_most(l), 0.0f) : warp_most(l);
  if (id >= 0) {
    const float e = expf(l - high);
    w = !p.sigmoid ? e * inv_sum : l > 0.0f ? __fdividef(1.0f, 1.0f + expf(-l)) : __fdividef(e, 1.0f + expf(l));
  }
  if (p.renormalize) {
    const float total = warp_sum(w);
    if (id >= 0) w = __fdividef(w, total);
  }
  if (lane < p.top_k) {
    const int64_t at = row * p.top_k + lane;
    if (MXFP4_IN_BOUNDS(p, kDbgIds, p.ids + at, 4)) p.ids[at] = id;
    if (MXFP4_IN_BOUNDS(p, kDbgWeights, p.weights + at, 4)) p.weights[at] = w * p.scale;
  }
}

template <int kPer, int kVec, LogitType kType>
cudaError_t launch_per(const TopkParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  const size_t words = warp_words(p.E, kPer == 0 || p.groups > 1);
  if (kPer == 0)
    if (const cudaError_t e = allow_smem(moe_topk_kernel<kPer, kVec, kType>,
                                         kWarps * warp_words(MXFP4_ROUTE_MAX_EXPERTS, true) * 4, ready);
        e != cudaSuccess)
      return e;
  return launch_pdl(moe_topk_kernel<kPer, kVec, kType>, dim3((p.tokens + kWarps - 1) / kWarps), kThreads,
                    kWarps * words * 4, stream, p);
}

template <LogitType kType>
cudaError_t launch_type(const TopkParams& p, cudaStream_t stream) {
  // four experts to a load where every row and the biases allow it
  const int size = kType == LogitType::kF32 ? 4 : 2;
  const bool wide = p.E % 4 == 0 && p.ld % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (4 * size) == 0 &&
                    reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
  // the fewest registers that hold a lane's keys
  if (p.E <= 4 * 32) return wide ? launch_per<4, 4, kType>(p, stream) : launch_per<4, 1, kType>(p, stream);
  if (p.E <= 12 * 32) return wide ? launch_per<12, 4, kType>(p, stream) : launch_per<12, 1, kType>(p, stream);
  if (p.E <= kMaxPerLane * 32)
    return wide ? launch_per<kMaxPerLane, 4, kType>(p, stream) : launch_per<kMaxPerLane, 1, kType>(p, stream);
  return launch_per<0, 1, kType>(p, stream);
}

}  // namespace

cudaError_t launch_moe_topk(const TopkArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  TopkParams p{};
  p.logits = a.logits;
  p.bias = a.bias;
  p.ids = a.ids;
  p.weights = a.weights;
  p.ld = a.ld;
  p.tokens = static_cast<int32_t>(a.num_tokens);
  p.E = a.E;
  p.groups = a.groups;
  p.size = a.E / a.groups;
  p.inv_size = 1.0f / static_cast<float>(p.size);
  p.top_groups = a.top_groups;
  p.top_k = a.top_k;
  p.scale = a.scale;
  p.sigmoid = a.sigmoid;
  p.group_sum2 = a.group_sum2;
  p.renormalize = a.renormalize;
  p.scored = a.bias != nullptr || (a.groups > 1 && a.group_sum2);
#ifdef MXFP4_DEBUG_BOUNDS
  debug_range(p.dbg, kDbgLogits, a.logits,
              ((a.num_tokens - 1) * a.ld + a.E) * (a.type == LogitType::kF32 ? 4 : 2));
  debug_range(p.dbg, kDbgBias, a.bias, a.bias ? a.E * 4 : 0);
  debug_range(p.dbg, kDbgIds, a.ids, a.num_tokens * a.top_k * 4);
  debug_range(p.dbg, kDbgWeights, a.weights, a.num_tokens * a.top_k * 4);
#endif
  if (a.type == LogitType::kF32) return launch_type<LogitType::kF32>(p, stream);
  return a.type == LogitType::kF16 ? launch_type<LogitType::kF16>(p, stream)
                                   : launch_type<LogitType::kBf16>(p, stream);
}

#ifdef MXFP4_DEBUG_BOUNDS
unsigned int debug_violations_topk() {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_debug_violations, sizeof v);
  cudaMemcpyToSymbol(g_debug_violations, &zero, sizeof zero);
  return v;
}
#endif

}  // namespace mxfp4

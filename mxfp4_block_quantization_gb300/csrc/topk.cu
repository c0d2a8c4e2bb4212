// topk.cu — the router's choice for sm_103a: the top_k experts of every token
// and their weights (formulas in include/mxfp4.h).
//
// A warp to a token; lane l holds the picks of experts l, l + 32, ... as 32-bit
// keys whose unsigned order is the picks' order (0: out), so a round of the
// choice is one redux.max over the lanes' best keys and one redux.min over the
// indices that have it: equal picks go to the lowest index.  Only the lane that
// lost its best looks through its keys again.
//
// Without a bias and group sums the keys are the logits, and exact.  Else they
// are float32 scores plus bias, and two closer than their error may be in the
// wrong order.  The choice notes the gaps between neighbours in its order, one
// beyond the last chosen; where a gap is within twice the error bound (about one
// token in 500 with 384 experts of ordinary spread) the token is chosen again by
// choose_exactly, which compares what is near in 64 bits.
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

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Unsigned keys in the order of finite floats, -0 with +0; none of them is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}
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
  const float s = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __expf(l - top) * inv_sum;
  return s + b;
}
// Twice what two neighbours of at most `m` may be off by together.
__device__ __forceinline__ float tolerance(const TopkParams& p, float m) {
  return (p.sigmoid ? 0x1p-20f : 0x1p-18f + 0x1p-27f * p.E) + 0x1p-21f * fabsf(m);
}

// The lanes' keys, in registers or (kPer == 0) in shared memory.
template <int kPer>
struct Keys {
  uint32_t v[kPer];
  __device__ __forceinline__ uint32_t get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(int i, uint32_t k) { v[i] = k; }
  __device__ __forceinline__ int count() const { return kPer; }
};
template <>
struct Keys<0> {
  uint32_t* v;
  int n;
  __device__ __forceinline__ uint32_t get(int i) const { return v[i * 32]; }
  __device__ __forceinline__ void set(int i, uint32_t k) { v[i * 32] = k; }
  __device__ __forceinline__ int count() const { return n; }
};

// ---------------------------------------------------- the exact choice
struct Exact {
  int64_t row;
  float top;        // the largest logit, and in float32 and 64 bits the softmax's
  float inv_sum;    // sum's inverse
  double sum;
  uint32_t kept;    // groups that stay
  uint32_t* gone;   // a bit for each expert that has been taken
};

__device__ __forceinline__ double pick64(const TopkParams& p, const Exact& x, float l, float b) {
  const double s = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
                             : exp(static_cast<double>(l) - x.top) / x.sum;
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
           ((x.kept >> (e / p.size)) & 1u);
  };
  uint32_t most = 0;
  for (int e = lo + lane; e < hi; e += 32) {
    float l, b, v;
    if (pick_at(e, l, b, v)) most = max(most, key_of(v));
  }
  most = __reduce_max_sync(kAll, most);
  if (most == 0) return -1;
  const float from = value_of(most) - tolerance(p, value_of(most));
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

// Lane j's chosen expert (-1: none), compared in 64 bits.
template <LogitType kType>
__device__ __noinline__ int choose_exactly(const TopkParams& p, int64_t row, float top,
                                           float inv_sum, uint32_t* gone) {
  const int lane = threadIdx.x & 31;
  Exact x{row, top, inv_sum, 1.0, kAll, gone};
  for (int i = lane; i < (p.E + 31) / 32; i += 32) gone[i] = 0;
  __syncwarp();
  if (!p.sigmoid) {
    double sum = 0.0;
    for (int e = lane; e < p.E; e += 32) {
      const float l = logit_at<kType>(p, row, e);
      if (finite(l)) sum += exp(static_cast<double>(l) - top);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    x.sum = sum;
  }
  const auto take = [&](int e) {
    if (lane == 0) gone[e >> 5] |= 1u << (e & 31);
    __syncwarp();
  };
  double value;
  if (p.groups > 1) {
    double mine = 0.0;
    bool open = false;
    for (int g = 0; g < p.groups; ++g) {
      const int lo = g * p.size, hi = lo + p.size;
      const int first = best_exactly<kType>(p, x, lo, hi, value);
      double total = value;
      if (first >= 0 && p.group_sum2) {
        take(first);
        if (best_exactly<kType>(p, x, lo, hi, value) >= 0) total += value;
      }
      if (lane == g) mine = total, open = first >= 0;
    }
    __syncwarp();
    for (int i = lane; i < (p.E + 31) / 32; i += 32) gone[i] = 0;
    __syncwarp();
    uint32_t kept = 0;
    for (int j = 0; j < p.top_groups; ++j) {
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
    x.kept = kept;
  }
  int id = -1;
  for (int j = 0; j < p.top_k; ++j) {
    const int e = best_exactly<kType>(p, x, 0, p.E, value);
    if (e < 0) break;
    if (lane == j) id = e;
    take(e);
  }
  return id;
}

// ------------------------------------------------------------ the kernel
template <int kPer, LogitType kType>
__global__ void __launch_bounds__(kThreads) moe_topk_kernel(const TopkParams p) {
  extern __shared__ uint32_t s_words[];  // per warp: E picks (groups or kPer == 0), E bits
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int padded = (p.E + 31) / 32 * 32;
  const bool in_smem = kPer == 0 || p.groups > 1;
  uint32_t* picks = s_words + static_cast<size_t>(warp) * ((in_smem ? padded : 0) + padded / 32);
  uint32_t* gone = picks + (in_smem ? padded : 0);
  pdl_wait();
  pdl_release();
  if (row >= p.tokens) return;

  // the logits, and the keys
  Keys<kPer> keys;
  if constexpr (kPer == 0) keys.v = picks + lane, keys.n = padded / 32;
  float top = -INFINITY, inv_sum = 1.0f;
  const bool softmax = !p.sigmoid;
#pragma unroll
  for (int i = 0; i < keys.count(); ++i) {
    const int e = i * 32 + lane;
    const float l = e < p.E ? logit_at<kType>(p, row, e) : INFINITY;
    keys.set(i, finite(l) ? key_of(l) : 0u);
    if (finite(l)) top = fmaxf(top, l);
  }
  if (softmax) {
    top = warp_max(top);
    if (p.scored || !p.renormalize) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < keys.count(); ++i) {
        const uint32_t k = keys.get(i);
        if (k != 0) sum += expf(value_of(k) - top);
      }
      inv_sum = 1.0f / warp_sum(sum);
    }
  }
  if (p.scored) {
#pragma unroll
    for (int i = 0; i < keys.count(); ++i) {
      const int e = i * 32 + lane;
      const uint32_t k = keys.get(i);
      const float b = e < p.E ? bias_at(p, e) : 0.0f;
      keys.set(i, k != 0 && finite(b) ? key_of(pick32(p, value_of(k), b, top, inv_sum)) : 0u);
    }
  }

  bool near = false;  // two neighbours in the order closer than their errors
  if (p.groups > 1) {
    if constexpr (kPer > 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 32 < padded) picks[i * 32 + lane] = keys.get(i);
    }
    __syncwarp();
    // 32 / share lanes to a group, its two best merged over them
    int share = 1;
    while (share < p.groups) share <<= 1;
    const int lanes = 32 / share;
    const int g = lane / lanes;
    uint32_t a = 0, b = 0;
    if (g < p.groups)
      for (int i = lane % lanes; i < p.size; i += lanes) {
        const uint32_t k = picks[g * p.size + i];
        b = max(b, min(a, k));
        a = max(a, k);
      }
    for (int d = lanes >> 1; d > 0; d >>= 1) {
      const uint32_t oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    float value = a ? value_of(a) : 0.0f, size = fabsf(value);
    if (p.group_sum2 && b) size += fabsf(value_of(b)), value += value_of(b);
    uint32_t key = a != 0 && g < p.groups && lane % lanes == 0 ? key_of(value) : 0u;
    const float tol = 2.0f * tolerance(p, p.scored ? warp_max(size) : 0.0f);
    uint32_t kept = 0;
    float last = 0.0f;
    for (int j = 0; j <= p.top_groups; ++j) {
      const uint32_t m = __reduce_max_sync(kAll, key);
      if (m == 0) break;
      if (j > 0) near |= last - value_of(m) <= tol;
      last = value_of(m);
      if (j == p.top_groups) break;
      const int at = __ffs(__ballot_sync(kAll, key == m)) - 1;
      kept |= 1u << (at / lanes);
      if (lane == at) key = 0;
    }
#pragma unroll
    for (int i = 0; i < keys.count(); ++i) {
      const int e = i * 32 + lane;
      if (e < p.E && !((kept >> (e / p.size)) & 1u)) keys.set(i, 0u);
    }
  }

  // the rounds
  int id = -1;
  uint32_t best = 0;
  int best_i = 0;
  const auto look = [&] {
    best = 0;
#pragma unroll
    for (int i = 0; i < keys.count(); ++i)
      if (keys.get(i) > best) best = keys.get(i), best_i = i;
  };
  look();
  float last = 0.0f;
  const int rounds = p.top_k + (p.scored ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0) break;
    if (j > 0) near |= last - value_of(m) <= tolerance(p, last);
    last = value_of(m);
    if (j == p.top_k) break;
    const int mine = best == m ? best_i * 32 + lane : INT32_MAX;
    const int e = __reduce_min_sync(kAll, mine);
    if (lane == j) id = e;
    if (mine == e) {
#pragma unroll
      for (int i = 0; i < keys.count(); ++i)
        if (i == best_i) keys.set(i, 0u);
      look();
    }
  }
  if (p.scored && near) id = choose_exactly<kType>(p, row, top, inv_sum, gone);

  // the weights, from the chosen logits (a renormalised softmax is the chosen
  // ones' own; small sigmoids are raised together, so that they do not vanish)
  float w = 0.0f;
  const float l = id >= 0 ? logit_at<kType>(p, row, id) : -INFINITY;
  float high = p.sigmoid ? 0.0f : top;
  if (p.renormalize) high = p.sigmoid ? fminf(warp_max(l), 0.0f) : warp_max(l);
  if (id >= 0) {
    const float e = expf(l - high);
    w = !p.sigmoid ? e * inv_sum : l > 0.0f ? 1.0f / (1.0f + expf(-l)) : e / (1.0f + expf(l));
  }
  if (p.renormalize) {
    const float total = warp_sum(w);
    if (id >= 0) w = w / total;
  }
  if (lane < p.top_k) {
    const int64_t at = row * p.top_k + lane;
    if (MXFP4_IN_BOUNDS(p, kDbgIds, p.ids + at, 4)) p.ids[at] = id;
    if (MXFP4_IN_BOUNDS(p, kDbgWeights, p.weights + at, 4)) p.weights[at] = w * p.scale;
  }
}

template <int kPer, LogitType kType>
cudaError_t launch_per(const TopkParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  const int padded = (p.E + 31) / 32 * 32;
  const size_t words = (kPer == 0 || p.groups > 1 ? padded : 0) + padded / 32;
  const size_t bytes = kWarps * words * 4;
  if (kPer == 0)
    if (const cudaError_t e = allow_smem(moe_topk_kernel<kPer, kType>,
                                         kWarps * (MXFP4_ROUTE_MAX_EXPERTS + MXFP4_ROUTE_MAX_EXPERTS / 32) * 4, ready);
        e != cudaSuccess)
      return e;
  return launch_pdl(moe_topk_kernel<kPer, kType>, dim3((p.tokens + kWarps - 1) / kWarps), kThreads,
                    bytes, stream, p);
}

template <LogitType kType>
cudaError_t launch_type(const TopkParams& p, cudaStream_t stream) {
  // the fewest registers that hold a lane's keys
  if (p.E <= 4 * 32) return launch_per<4, kType>(p, stream);
  if (p.E <= 8 * 32) return launch_per<8, kType>(p, stream);
  if (p.E <= 12 * 32) return launch_per<12, kType>(p, stream);
  if (p.E <= kMaxPerLane * 32) return launch_per<kMaxPerLane, kType>(p, stream);
  return launch_per<0, kType>(p, stream);
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

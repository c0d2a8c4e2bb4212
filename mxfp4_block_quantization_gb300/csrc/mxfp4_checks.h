// mxfp4_checks.h — host-side argument checks shared by the C entry points
// (mxfp4_api.cu, mxfp4_decode_api.cu).
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/mxfp4.h"

namespace mxfp4 {
namespace checks {

constexpr int64_t kMaxGrid = INT_MAX / 2;  // tile counts stay far from int overflow

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + static_cast<uintptr_t>(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ECUDA; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int64_t padded_scale_cols(int64_t K) { return ceil_div(K / 32, 4) * 4; }

// Byte count of `rows` rows of `cols` scale bytes for a size query, or 0 when
// it does not fit in int64 (no call accepts such sizes).
inline size_t rows_times_cols(int64_t rows, int64_t cols) {
  int64_t r = 0;
  return __builtin_mul_overflow(rows, cols, &r) ? 0 : static_cast<size_t>(r);
}

// Row counts above this are rejected by every call; the size queries return
// 0 for them instead of wrapping around.
constexpr int64_t kMaxRows = INT64_MAX / 4;

}  // namespace checks
}  // namespace mxfp4

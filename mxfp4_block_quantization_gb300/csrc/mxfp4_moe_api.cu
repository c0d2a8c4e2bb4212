// mxfp4_moe_api.cu — the extern "C" entry points of a layer's products over
// many tokens: the router's choice, products of quantized activations with
// quantized weights (dense and per expert) and the experts' rows back to their
// tokens.  Host-side checks only, then the launchers; see include/mxfp4.h.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "mxfp4_checks.h"
#include "mxfp4_internal.h"
#include "../../include/mxfp4.h"

namespace {

using namespace mxfp4::checks;

int topk_checked(const mxfp4::TopkArgs& a, int32_t score, int32_t group_sum2, int32_t renormalize,
                 void* stream) {
  if (a.num_tokens < 0 || a.E < 1 || a.top_k < 1 || a.groups < 1 || a.top_groups < 1 ||
      (score != MXFP4_SCORE_SOFTMAX && score != MXFP4_SCORE_SIGMOID) ||
      (group_sum2 != 0 && group_sum2 != 1) || (renormalize != 0 && renormalize != 1) ||
      !std::isfinite(a.scale))
    return MXFP4_EINVAL;
  if (a.E > MXFP4_ROUTE_MAX_EXPERTS || a.top_k > a.E || a.top_k > MXFP4_TOPK_MAX ||
      a.groups > 32 || a.E % a.groups != 0 || a.top_groups > a.groups || a.ld < a.E ||
      a.num_tokens > INT32_MAX / 2)
    return MXFP4_ESHAPE;
  if (a.num_tokens > 0 && a.ld > (INT64_MAX / 8) / a.num_tokens) return MXFP4_ESHAPE;
  if (a.num_tokens > 0 && (!a.logits || !a.ids || !a.weights)) return MXFP4_EINVAL;
  const int size = a.type == mxfp4::LogitType::kF32 ? 4 : 2;
  if (!aligned_to(a.logits, static_cast<uintptr_t>(size)) || !aligned_to(a.bias, 4) ||
      !aligned_to(a.ids, 4) || !aligned_to(a.weights, 4))
    return MXFP4_EALIGN;
  const int64_t out = a.num_tokens * a.top_k * 4;
  const Range ins[2] = {
      range_of(a.logits, a.num_tokens > 0 ? ((a.num_tokens - 1) * a.ld + a.E) * size : 0),
      range_of(a.bias, a.bias ? static_cast<int64_t>(a.E) * 4 : 0)};
  const Range outs[2] = {range_of(a.ids, out), range_of(a.weights, out)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return MXFP4_EALIAS;
  if (overlap(outs[0], outs[1])) return MXFP4_EALIAS;
  return from_cuda(mxfp4::launch_moe_topk(a, static_cast<cudaStream_t>(stream)));
}

int topk(const void* logits, mxfp4::LogitType type, int64_t T, int32_t E, int64_t ld,
         const float* bias, int32_t score, int32_t groups, int32_t top_groups, int32_t group_sum2,
         int32_t top_k, int32_t renormalize, float scale, int32_t* ids, float* weights,
         void* stream) {
  mxfp4::TopkArgs a{};
  a.logits = logits;
  a.type = type;
  a.num_tokens = T;
  a.E = E;
  a.ld = ld;
  a.bias = bias;
  a.sigmoid = score == MXFP4_SCORE_SIGMOID;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_sum2 = group_sum2 == 1;
  a.top_k = top_k;
  a.renormalize = renormalize == 1;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  return topk_checked(a, score, group_sum2, renormalize, stream);
}

// y and an input of the same rows: apart, or the very same elements.
bool clash(const void* y, int64_t ldy, Range out, const void* in, int64_t ld, Range range) {
  return overlap(out, range) && !(y == in && ldy == ld);
}

int gemm_checked(const mxfp4::GemmArgs& a, bool moe, void* stream) {
  if (a.rows < 0 || a.K < 0 || a.N < 0 || a.E < 0 || a.activation < MXFP4_ACT_NONE ||
      a.activation > MXFP4_ACT_GELU_TANH || a.gate < MXFP4_GATE_NONE ||
      a.gate > MXFP4_GATE_SECOND)
    return MXFP4_EINVAL;
  const bool gated = a.gate != MXFP4_GATE_NONE;
  if (a.K % 32 != 0 || (gated && a.N % 2 != 0)) return MXFP4_ESHAPE;
  const int64_t cols = gated ? a.N / 2 : a.N;
  if (a.ldy < cols || (a.residual && a.ldr < cols)) return MXFP4_ESHAPE;
  if (moe) {
    if (!a.offsets) return MXFP4_EINVAL;
    if (a.E == 0 && a.rows > 0) return MXFP4_EINVAL;
    if (a.E > MXFP4_ROUTE_MAX_EXPERTS) return MXFP4_ESHAPE;
  }
  const bool work = a.rows > 0 && cols > 0 && a.E > 0;
  const bool reads = work && a.K > 0;
  if (work && !a.y) return MXFP4_EINVAL;
  if (reads && (!a.x_codes || !a.x_scales || !a.codes || !a.scales)) return MXFP4_EINVAL;
  if (reads && a.nvfp4 && (!a.x_globals || !a.globals)) return MXFP4_EINVAL;
  if (!work && !moe) return MXFP4_OK;
  // rows, weight rows of all experts, tiles and K are counted in int32, bytes in int64
  if (a.K > INT32_MAX / 2 || a.rows > INT32_MAX / 2 || (a.E > 0 && a.N > (INT32_MAX / 2) / a.E))
    return MXFP4_ESHAPE;
  if ((a.rows / 128 + a.E + 1) > INT32_MAX / (a.N / 128 + 2)) return MXFP4_ESHAPE;
  if (a.rows > 0 && (a.ldy > (INT64_MAX / 8) / a.rows || (a.residual && a.ldr > (INT64_MAX / 8) / a.rows)))
    return MXFP4_ESHAPE;
  const int64_t w_scales = static_cast<int64_t>(a.nvfp4 ? mxfp4_nvfp4_scale_bytes(a.N, a.K)
                                                        : mxfp4_scale_bytes(a.N, a.K));
  const int64_t x_scales = static_cast<int64_t>(
      moe ? (a.nvfp4 ? mxfp4_nvfp4_grouped_scale_bytes_bound(a.rows, a.E, a.K)
                     : mxfp4_grouped_scale_bytes_bound(a.rows, a.E, a.K))
          : (a.nvfp4 ? mxfp4_nvfp4_scale_bytes(a.rows, a.K) : mxfp4_scale_bytes(a.rows, a.K)));
  if (!aligned16(a.x_codes) || !aligned16(a.x_scales) || !aligned16(a.codes) ||
      !aligned16(a.scales) || !aligned_to(a.x_globals, 4) || !aligned_to(a.globals, 4) ||
      !aligned_to(a.offsets, 4) || !aligned_to(a.bias, 2) || !aligned_to(a.residual, 2) ||
      !aligned_to(a.y, 2) || !aligned_to(a.status, 4))
    return MXFP4_EALIGN;
  const Range residual = range_of(a.residual, a.residual && work ? ((a.rows - 1) * a.ldr + cols) * 2 : 0);
  const Range ins[8] = {
      range_of(a.x_codes, reads ? a.rows * (a.K / 2) : 0), range_of(a.x_scales, reads ? x_scales : 0),
      range_of(a.codes, reads ? a.E * a.N * (a.K / 2) : 0), range_of(a.scales, reads ? a.E * w_scales : 0),
      range_of(a.x_globals, a.nvfp4 && reads ? a.E * 4 : 0),
      range_of(a.globals, a.nvfp4 && reads ? a.E * 4 : 0),
      range_of(a.bias, a.bias && work ? a.E * a.N * 2 : 0),
      range_of(a.offsets, moe ? (static_cast<int64_t>(a.E) + 1) * 4 : 0)};
  const Range outs[2] = {range_of(a.y, work ? ((a.rows - 1) * a.ldy + cols) * 2 : 0),
                         range_of(a.status, a.status ? 4 : 0)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return MXFP4_EALIAS;
  if (overlap(outs[0], outs[1]) || overlap(outs[1], residual) ||
      clash(a.y, a.ldy, outs[0], a.residual, a.ldr, residual))
    return MXFP4_EALIAS;
  return from_cuda(mxfp4::launch_gemm(a, static_cast<cudaStream_t>(stream)));
}

mxfp4::GemmArgs gemm_args(const uint8_t* x_codes, const uint8_t* x_scales, const float* xg,
                          int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales,
                          const float* g, int64_t N, const void* bias, int32_t activation,
                          int32_t gate, void* y, int64_t ldy, bool f16, bool nvfp4) {
  mxfp4::GemmArgs a{};
  a.x_codes = x_codes;
  a.x_scales = x_scales;
  a.x_globals = xg;
  a.rows = rows;
  a.K = K;
  a.E = 1;
  a.codes = codes;
  a.scales = scales;
  a.globals = g;
  a.N = N;
  a.bias = bias;
  a.activation = activation;
  a.gate = gate;
  a.y = y;
  a.ldy = ldy;
  a.f16 = f16;
  a.nvfp4 = nvfp4;
  return a;
}

int dense(mxfp4::GemmArgs a, const void* residual, int64_t ldr, void* stream) {
  a.residual = residual;
  a.ldr = ldr;
  return gemm_checked(a, false, stream);
}

int moe(mxfp4::GemmArgs a, const int32_t* offsets, int32_t E, int32_t* status, void* stream) {
  a.offsets = offsets;
  a.E = E;
  a.status = status;
  return gemm_checked(a, true, stream);
}

int combine_checked(const mxfp4::CombineArgs& a, int32_t rows_f32, void* stream) {
  if (a.total_rows < 0 || a.N < 0 || a.num_tokens < 0 || a.top_k < 1 ||
      (rows_f32 != 0 && rows_f32 != 1))
    return MXFP4_EINVAL;
  if (a.ldr < a.N || a.ldy < a.N || (a.residual && a.ld_res < a.N)) return MXFP4_ESHAPE;
  // routes and threads (a column each at worst) are counted in int32
  if (a.num_tokens > (INT32_MAX / 2) / a.top_k || a.N > INT32_MAX / 2 || a.total_rows > INT32_MAX ||
      (a.N > 0 && a.num_tokens > kMaxGrid / ((a.N + 255) / 256)))
    return MXFP4_ESHAPE;
  const int size = a.rows_f32 ? 4 : 2;
  if ((a.total_rows > 0 && a.ldr > (INT64_MAX / 8) / a.total_rows) ||
      (a.num_tokens > 0 && (a.ldy > (INT64_MAX / 8) / a.num_tokens ||
                            (a.residual && a.ld_res > (INT64_MAX / 8) / a.num_tokens))))
    return MXFP4_ESHAPE;
  const bool work = a.num_tokens > 0 && a.N > 0;
  if (a.num_tokens > 0 && !a.dest) return MXFP4_EINVAL;
  if (work && (!a.weights || !a.y || (a.total_rows > 0 && !a.rows))) return MXFP4_EINVAL;
  if (!aligned_to(a.rows, static_cast<uintptr_t>(size)) || !aligned_to(a.dest, 4) ||
      !aligned_to(a.weights, 4) || !aligned_to(a.residual, 2) || !aligned_to(a.y, 2) ||
      !aligned_to(a.status, 4))
    return MXFP4_EALIGN;
  const int64_t routes = a.num_tokens * a.top_k * 4;
  const Range residual = range_of(a.residual, a.residual && work ? ((a.num_tokens - 1) * a.ld_res + a.N) * 2 : 0);
  const Range ins[3] = {
      range_of(a.rows, work && a.total_rows > 0 ? ((a.total_rows - 1) * a.ldr + a.N) * size : 0),
      range_of(a.dest, routes), range_of(a.weights, work ? routes : 0)};
  const Range outs[2] = {range_of(a.y, work ? ((a.num_tokens - 1) * a.ldy + a.N) * 2 : 0),
                         range_of(a.status, a.status ? 4 : 0)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return MXFP4_EALIAS;
  if (overlap(outs[0], outs[1]) || overlap(outs[1], residual) ||
      clash(a.y, a.ldy, outs[0], a.residual, a.ld_res, residual))
    return MXFP4_EALIAS;
  return from_cuda(mxfp4::launch_moe_combine(a, static_cast<cudaStream_t>(stream)));
}

int combine(const void* rows, int32_t rows_f32, int64_t total_rows, int64_t N, int64_t ldr,
            const int32_t* dest, const float* weights, int64_t T, int32_t top_k,
            const void* residual, int64_t ld_res, void* y, int64_t ldy, int32_t* status, bool f16,
            void* stream) {
  mxfp4::CombineArgs a{};
  a.rows = rows;
  a.rows_f32 = rows_f32 == 1;
  a.total_rows = total_rows;
  a.N = N;
  a.ldr = ldr;
  a.dest = dest;
  a.weights = weights;
  a.num_tokens = T;
  a.top_k = top_k;
  a.residual = residual;
  a.ld_res = ld_res;
  a.y = y;
  a.ldy = ldy;
  a.status = status;
  a.f16 = f16;
  return combine_checked(a, rows_f32, stream);
}

}  // namespace

extern "C" {

#define MXFP4_TOPK(name, type)                                                                   \
  int name(const void* logits, int64_t num_tokens, int32_t E, int64_t ld, const float* bias,     \
           int32_t score, int32_t groups, int32_t top_groups, int32_t group_sum2, int32_t top_k, \
           int32_t renormalize, float scale, int32_t* ids, float* weights, void* stream) {       \
    return topk(logits, type, num_tokens, E, ld, bias, score, groups, top_groups, group_sum2,    \
                top_k, renormalize, scale, ids, weights, stream);                                \
  }
MXFP4_TOPK(mxfp4_moe_topk, mxfp4::LogitType::kBf16)
MXFP4_TOPK(mxfp4_moe_topk_f16, mxfp4::LogitType::kF16)
MXFP4_TOPK(mxfp4_moe_topk_f32, mxfp4::LogitType::kF32)
#undef MXFP4_TOPK

#define MXFP4_GEMM(name, f16)                                                                     \
  int name(const uint8_t* x_codes, const uint8_t* x_scales, int64_t num_tokens, int64_t K,        \
           const uint8_t* codes, const uint8_t* scales, int64_t N, const void* bias,              \
           int32_t activation, int32_t gate, const void* residual, int64_t ldr, void* y,          \
           int64_t ldy, void* stream) {                                                           \
    return dense(gemm_args(x_codes, x_scales, nullptr, num_tokens, K, codes, scales, nullptr, N,  \
                           bias, activation, gate, y, ldy, f16, false),                           \
                 residual, ldr, stream);                                                          \
  }
MXFP4_GEMM(mxfp4_gemm, false)
MXFP4_GEMM(mxfp4_gemm_f16, true)
#undef MXFP4_GEMM

#define MXFP4_GEMM_NVFP4(name, f16)                                                               \
  int name(const uint8_t* x_codes, const uint8_t* x_scales, const float* x_global_scale,          \
           int64_t num_tokens, int64_t K, const uint8_t* codes, const uint8_t* scales,            \
           const float* global_scale, int64_t N, const void* bias, int32_t activation,            \
           int32_t gate, const void* residual, int64_t ldr, void* y, int64_t ldy, void* stream) { \
    return dense(gemm_args(x_codes, x_scales, x_global_scale, num_tokens, K, codes, scales,       \
                           global_scale, N, bias, activation, gate, y, ldy, f16, true),           \
                 residual, ldr, stream);                                                          \
  }
MXFP4_GEMM_NVFP4(mxfp4_gemm_nvfp4, false)
MXFP4_GEMM_NVFP4(mxfp4_gemm_nvfp4_f16, true)
#undef MXFP4_GEMM_NVFP4

#define MXFP4_MOE_GEMM(name, f16)                                                                \
  int name(const uint8_t* x_codes, const uint8_t* x_scales, int64_t total_rows, int64_t K,       \
           const int32_t* expert_offsets, int32_t E, const uint8_t* codes, const uint8_t* scales, \
           int64_t N, const void* bias, int32_t activation, int32_t gate, void* y, int64_t ldy,  \
           int32_t* status, void* stream) {                                                      \
    return moe(gemm_args(x_codes, x_scales, nullptr, total_rows, K, codes, scales, nullptr, N,   \
                         bias, activation, gate, y, ldy, f16, false),                            \
               expert_offsets, E, status, stream);                                               \
  }
MXFP4_MOE_GEMM(mxfp4_moe_gemm, false)
MXFP4_MOE_GEMM(mxfp4_moe_gemm_f16, true)
#undef MXFP4_MOE_GEMM

#define MXFP4_MOE_GEMM_NVFP4(name, f16)                                                          \
  int name(const uint8_t* x_codes, const uint8_t* x_scales, const float* x_global_scales,        \
           int64_t total_rows, int64_t K, const int32_t* expert_offsets, int32_t E,              \
           const uint8_t* codes, const uint8_t* scales, const float* global_scales, int64_t N,   \
           const void* bias, int32_t activation, int32_t gate, void* y, int64_t ldy,             \
           int32_t* status, void* stream) {                                                      \
    return moe(gemm_args(x_codes, x_scales, x_global_scales, total_rows, K, codes, scales,       \
                         global_scales, N, bias, activation, gate, y, ldy, f16, true),           \
               expert_offsets, E, status, stream);                                               \
  }
MXFP4_MOE_GEMM_NVFP4(mxfp4_moe_gemm_nvfp4, false)
MXFP4_MOE_GEMM_NVFP4(mxfp4_moe_gemm_nvfp4_f16, true)
#undef MXFP4_MOE_GEMM_NVFP4

#define MXFP4_COMBINE(name, f16)                                                                 \
  int name(const void* rows, int32_t rows_f32, int64_t total_rows, int64_t N, int64_t ldr,       \
           const int32_t* dest_rows, const float* weights, int64_t num_tokens, int32_t top_k,    \
           const void* residual, int64_t ld_res, void* y, int64_t ldy, int32_t* status,          \
           void* stream) {                                                                       \
    return combine(rows, rows_f32, total_rows, N, ldr, dest_rows, weights, num_tokens, top_k,    \
                   residual, ld_res, y, ldy, status, f16, stream);                               \
  }
MXFP4_COMBINE(mxfp4_moe_combine, false)
MXFP4_COMBINE(mxfp4_moe_combine_f16, true)
#undef MXFP4_COMBINE

}  // extern "C"

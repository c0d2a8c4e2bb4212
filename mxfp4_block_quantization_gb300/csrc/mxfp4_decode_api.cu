// mxfp4_decode_api.cu — the extern "C" entry points of a decode step:
// products with 4-bit weights, the paged 4-bit cache and the attention over
// it.  Host-side checks only, then the launchers; see include/mxfp4.h.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "mxfp4_checks.h"
#include "mxfp4_internal.h"
#include "../../include/mxfp4.h"

namespace {

using namespace mxfp4::checks;

int matvec_checked(mxfp4::MatvecArgs a, int32_t y_f32, bool moe, void* stream) {
  const int64_t block = a.nvfp4 ? 16 : 32;
  if (a.src_rows < 0 || a.rows < 0 || a.K < 0 || a.N < 0 || a.E < 0 || (y_f32 != 0 && y_f32 != 1))
    return MXFP4_EINVAL;
  if (a.K % block != 0 || a.ldx < a.K || a.ldy < a.N) return MXFP4_ESHAPE;
  if (moe) {
    if (!a.offsets) return MXFP4_EINVAL;
    if (a.E == 0 && a.rows > 0) return MXFP4_EINVAL;
    if (a.E > MXFP4_ROUTE_MAX_EXPERTS || a.rows > INT32_MAX / 2 || a.src_rows > INT32_MAX)
      return MXFP4_ESHAPE;
    if (!a.row_index && a.src_rows < a.rows) return MXFP4_ESHAPE;
  }
  const bool work = a.rows > 0 && a.N > 0 && a.E > 0;
  const bool reads = work && a.K > 0;
  if (work && !a.y) return MXFP4_EINVAL;
  if (reads && (!a.codes || !a.scales || (a.src_rows > 0 && !a.x))) return MXFP4_EINVAL;
  if (reads && a.nvfp4 && !a.global_scales) return MXFP4_EINVAL;
  if (!work && !moe) return MXFP4_OK;
  a.y_f32 = y_f32 == 1;
  const int64_t size = a.y_f32 ? 4 : 2;
  // byte counts stay inside int64, K and the row-tile counts inside int32
  const int64_t scale_bytes = static_cast<int64_t>(a.nvfp4 ? mxfp4_nvfp4_scale_bytes(a.N, a.K)
                                                           : mxfp4_scale_bytes(a.N, a.K));
  if (a.K > INT32_MAX / 2 || a.N > kMaxGrid || a.rows > kMaxGrid) return MXFP4_ESHAPE;
  if (a.src_rows > 0 && a.ldx > (INT64_MAX / 4) / a.src_rows) return MXFP4_ESHAPE;
  if (a.rows > 0 && a.ldy > (INT64_MAX / 8) / a.rows) return MXFP4_ESHAPE;
  // units of 8 or more rows by 16-row tiles of the weights, counted in int32
  if ((a.rows / 8 + a.E + 1) > INT32_MAX / (a.N / 16 + 8)) return MXFP4_ESHAPE;
  if (reads && a.N * (a.K / 2) > (INT64_MAX / 4) / a.E) return MXFP4_ESHAPE;
  if (!aligned16(a.x) || (reads && a.src_rows > 1 && a.ldx % 8 != 0) || !aligned16(a.codes) ||
      !aligned16(a.scales) || !aligned_to(a.y, static_cast<uintptr_t>(size)) ||
      !aligned_to(a.global_scales, 4) || !aligned_to(a.row_index, 4) ||
      !aligned_to(a.offsets, 4) || !aligned_to(a.status, 4))
    return MXFP4_EALIGN;
  const Range ins[6] = {
      range_of(a.x, a.src_rows > 0 ? ((a.src_rows - 1) * a.ldx + a.K) * 2 : 0),
      range_of(a.codes, reads ? a.E * a.N * (a.K / 2) : 0),
      range_of(a.scales, reads ? a.E * scale_bytes : 0),
      range_of(a.global_scales, a.nvfp4 && reads ? static_cast<int64_t>(a.E) * 4 : 0),
      range_of(a.row_index, a.row_index ? a.rows * 4 : 0),
      range_of(a.offsets, moe ? (static_cast<int64_t>(a.E) + 1) * 4 : 0)};
  const Range outs[2] = {range_of(a.y, work ? ((a.rows - 1) * a.ldy + a.N) * size : 0),
                         range_of(a.status, a.status ? 4 : 0)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return MXFP4_EALIAS;
  if (overlap(outs[0], outs[1])) return MXFP4_EALIAS;
  return from_cuda(mxfp4::launch_matvec(a, static_cast<cudaStream_t>(stream)));
}

int dense_matvec(const void* x, int64_t T, int64_t K, int64_t ldx, const uint8_t* codes,
                 const uint8_t* scales, const float* g, int64_t N, void* y, int64_t ldy,
                 int32_t y_f32, bool f16, bool nvfp4, void* stream) {
  mxfp4::MatvecArgs a{};
  a.x = x;
  a.src_rows = a.rows = T;
  a.K = K;
  a.ldx = ldx;
  a.E = 1;
  a.codes = codes;
  a.scales = scales;
  a.global_scales = g;
  a.N = N;
  a.y = y;
  a.ldy = ldy;
  a.f16 = f16;
  a.nvfp4 = nvfp4;
  return matvec_checked(a, y_f32, false, stream);
}

int moe_matvec(const void* x, int64_t src_rows, int64_t K, int64_t ldx, const int32_t* row_index,
               int64_t rows, const int32_t* offsets, int32_t E, const uint8_t* codes,
               const uint8_t* scales, const float* g, int64_t N, void* y, int64_t ldy,
               int32_t y_f32, int32_t* status, bool f16, bool nvfp4, void* stream) {
  mxfp4::MatvecArgs a{};
  a.x = x;
  a.src_rows = src_rows;
  a.K = K;
  a.ldx = ldx;
  a.row_index = row_index;
  a.rows = rows;
  a.offsets = offsets;
  a.E = E;
  a.codes = codes;
  a.scales = scales;
  a.global_scales = g;
  a.N = N;
  a.y = y;
  a.ldy = ldy;
  a.f16 = f16;
  a.nvfp4 = nvfp4;
  a.status = status;
  return matvec_checked(a, y_f32, true, stream);
}

// The cache's shape and its four tensors; `work` is whether the call touches
// them.  Fills bytes[0] (codes of keys or of values) and bytes[1] (scales).
int cache_checked(const mxfp4::CacheArgs& c, bool work, int64_t bytes[2]) {
  if (c.num_pages < 0 || c.page_size < 1 || c.num_heads < 0 || c.head_dim < 0) return MXFP4_EINVAL;
  if (c.head_dim % 32 != 0 || c.num_pages > INT32_MAX / c.page_size) return MXFP4_ESHAPE;
  const int64_t rows = c.num_pages * c.page_size;
  const int64_t row = static_cast<int64_t>(c.num_heads) * c.head_dim;
  if (row > INT32_MAX) return MXFP4_ESHAPE;
  bytes[0] = rows * (row / 2);
  bytes[1] = rows * (row / (c.nvfp4 ? 16 : 32));
  for (int i = 0; i < 2; ++i) {
    if (work && (!c.codes[i] || !c.scales[i] || (c.nvfp4 && !c.global_scales[i])))
      return MXFP4_EINVAL;
    if (!aligned16(c.codes[i]) || !aligned16(c.scales[i]) || !aligned_to(c.global_scales[i], 4))
      return MXFP4_EALIGN;
  }
  return MXFP4_OK;
}

mxfp4::CacheArgs cache_args(const uint8_t* kc, const uint8_t* ks, const uint8_t* vc,
                            const uint8_t* vs, const float* kg, const float* vg,
                            int64_t num_pages, int32_t page_size, int32_t num_heads,
                            int32_t head_dim, bool f16, bool nvfp4) {
  mxfp4::CacheArgs c{};
  c.codes[0] = const_cast<uint8_t*>(kc);
  c.codes[1] = const_cast<uint8_t*>(vc);
  c.scales[0] = const_cast<uint8_t*>(ks);
  c.scales[1] = const_cast<uint8_t*>(vs);
  c.global_scales[0] = kg;
  c.global_scales[1] = vg;
  c.num_pages = num_pages;
  c.page_size = page_size;
  c.num_heads = num_heads;
  c.head_dim = head_dim;
  c.f16 = f16;
  c.nvfp4 = nvfp4;
  return c;
}

// Strides of a [rows, heads, head_dim] input: both non-negative, in whole
// 16-byte pieces, and the last element's byte offset inside int64.
int strides_checked(const void* p, int64_t rows, int64_t heads, int64_t row_stride,
                    int64_t head_stride) {
  if (row_stride < 0 || head_stride < 0) return MXFP4_EINVAL;
  if (rows > 0 && row_stride > (INT64_MAX / 16) / rows) return MXFP4_ESHAPE;
  if (heads > 0 && head_stride > (INT64_MAX / 16) / heads) return MXFP4_ESHAPE;
  if (!aligned16(p) || row_stride % 8 != 0 || head_stride % 8 != 0) return MXFP4_EALIGN;
  return MXFP4_OK;
}

Range strided_range(const void* p, int64_t rows, int64_t heads, int64_t row_stride,
                    int64_t head_stride, int64_t head_dim) {
  if (rows <= 0 || heads <= 0 || head_dim <= 0) return range_of(p, 0);
  return range_of(p, ((rows - 1) * row_stride + (heads - 1) * head_stride + head_dim) * 2);
}

int write_checked(const mxfp4::CacheArgs& c, const void* k, const void* v, int64_t T,
                  int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                  int64_t v_head_stride, const int32_t* slots, int32_t* status, void* stream) {
  if (T < 0) return MXFP4_EINVAL;
  const bool work = T > 0 && c.num_heads > 0 && c.head_dim > 0;
  int64_t bytes[2];
  if (const int rc = cache_checked(c, work && c.num_pages > 0, bytes)) return rc;
  if (work && (!k || !v)) return MXFP4_EINVAL;
  if (T > 0 && !slots) return MXFP4_EINVAL;
  if (T > INT32_MAX || T * c.num_heads > kMaxGrid) return MXFP4_ESHAPE;
  if (const int rc = strides_checked(k, T, c.num_heads, k_token_stride, k_head_stride)) return rc;
  if (const int rc = strides_checked(v, T, c.num_heads, v_token_stride, v_head_stride)) return rc;
  if (!aligned_to(slots, 4) || !aligned_to(status, 4)) return MXFP4_EALIGN;
  const Range ins[5] = {
      strided_range(k, T, c.num_heads, k_token_stride, k_head_stride, c.head_dim),
      strided_range(v, T, c.num_heads, v_token_stride, v_head_stride, c.head_dim),
      range_of(slots, T * 4), range_of(c.global_scales[0], c.nvfp4 ? 4 : 0),
      range_of(c.global_scales[1], c.nvfp4 ? 4 : 0)};
  const Range outs[5] = {range_of(c.codes[0], bytes[0]), range_of(c.scales[0], bytes[1]),
                         range_of(c.codes[1], bytes[0]), range_of(c.scales[1], bytes[1]),
                         range_of(status, status ? 4 : 0)};
  for (int i = 0; i < 5; ++i) {
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return MXFP4_EALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (overlap(outs[i], outs[j])) return MXFP4_EALIAS;
  }
  const void* const x[2] = {k, v};
  const int64_t ts[2] = {k_token_stride, v_token_stride};
  const int64_t hs[2] = {k_head_stride, v_head_stride};
  return from_cuda(mxfp4::launch_cache_write(c, x, T, ts, hs, slots, status,
                                             static_cast<cudaStream_t>(stream)));
}

int read_checked(const mxfp4::CacheArgs& c, const int32_t* slots, int64_t T, void* k_out,
                 void* v_out, int32_t* status, void* stream) {
  if (T < 0) return MXFP4_EINVAL;
  const bool work = T > 0 && c.num_heads > 0 && c.head_dim > 0;
  int64_t bytes[2];
  if (const int rc = cache_checked(c, work && c.num_pages > 0, bytes)) return rc;
  if (work && (!k_out || !v_out)) return MXFP4_EINVAL;
  if (T > 0 && !slots) return MXFP4_EINVAL;
  if (T > INT32_MAX || T * c.num_heads > kMaxGrid) return MXFP4_ESHAPE;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned_to(slots, 4) || !aligned_to(status, 4))
    return MXFP4_EALIGN;
  const int64_t out_bytes = T * c.num_heads * c.head_dim * 2;
  const Range ins[7] = {range_of(c.codes[0], bytes[0]), range_of(c.scales[0], bytes[1]),
                        range_of(c.codes[1], bytes[0]), range_of(c.scales[1], bytes[1]),
                        range_of(slots, T * 4), range_of(c.global_scales[0], c.nvfp4 ? 4 : 0),
                        range_of(c.global_scales[1], c.nvfp4 ? 4 : 0)};
  const Range outs[3] = {range_of(k_out, out_bytes), range_of(v_out, out_bytes),
                         range_of(status, status ? 4 : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return MXFP4_EALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return MXFP4_EALIAS;
  }
  void* const out[2] = {k_out, v_out};
  return from_cuda(mxfp4::launch_cache_read(c, slots, T, out, status,
                                            static_cast<cudaStream_t>(stream)));
}

int attention_checked(const mxfp4::AttentionArgs& a, size_t workspace_bytes, void* stream) {
  const mxfp4::CacheArgs& c = a.cache;
  if (a.num_seqs < 0 || a.num_q_heads < 0 || a.max_pages < 0 || a.window < 0 ||
      a.table_stride < 0 || !std::isfinite(a.softmax_scale))
    return MXFP4_EINVAL;
  const bool work = a.num_seqs > 0 && a.num_q_heads > 0 && c.head_dim > 0;
  int64_t bytes[2];
  if (const int rc = cache_checked(c, work && c.num_pages > 0 && a.max_pages > 0, bytes)) return rc;
  if (c.head_dim > MXFP4_ATTENTION_MAX_HEAD_DIM || a.max_pages > INT32_MAX / c.page_size ||
      a.table_stride < a.max_pages || a.num_seqs > kMaxGrid)
    return MXFP4_ESHAPE;
  // the steps of all (sequence, kv head, 8 query heads) are counted in int32,
  // padded by at most a share of each; rows of the cache in uint32
  if (work && c.num_heads > 0) {
    const int64_t units = a.num_seqs * c.num_heads * ceil_div(a.num_q_heads / c.num_heads, 8);
    if (units > INT32_MAX / 2 / (a.max_pages * c.page_size / 32 + 1)) return MXFP4_ESHAPE;
  }
  if (c.num_heads > 0 && c.num_pages * c.page_size > static_cast<int64_t>(UINT32_MAX) / c.num_heads)
    return MXFP4_ESHAPE;
  if (a.num_q_heads > 0 && (c.num_heads == 0 || a.num_q_heads % c.num_heads != 0))
    return MXFP4_ESHAPE;
  if (work && (!a.q || !a.out)) return MXFP4_EINVAL;
  // without heads the status word still comes from the lengths and pages
  if ((work || (a.status && a.num_seqs > 0)) &&
      (!a.seq_lens || (a.max_pages > 0 && !a.page_table)))
    return MXFP4_EINVAL;
  if (a.num_q_heads > 0 && a.num_seqs > kMaxGrid / a.num_q_heads) return MXFP4_ESHAPE;
  if (a.num_seqs > 0 && a.table_stride > (INT64_MAX / 8) / a.num_seqs) return MXFP4_ESHAPE;
  if (const int rc = strides_checked(a.q, a.num_seqs, a.num_q_heads, a.q_seq_stride,
                                     a.q_head_stride))
    return rc;
  const int64_t ws_bytes =
      4 * mxfp4::attention_workspace_floats(a.num_seqs, a.num_q_heads, c.num_heads, c.head_dim,
                                            a.max_pages * c.page_size);
  if (work && ws_bytes > 0 && (!a.workspace || workspace_bytes < static_cast<size_t>(ws_bytes)))
    return MXFP4_EINVAL;
  if (!aligned16(a.workspace) || !aligned16(a.out) || !aligned_to(a.lse, 4) ||
      !aligned_to(a.page_table, 4) || !aligned_to(a.seq_lens, 4) || !aligned_to(a.status, 4))
    return MXFP4_EALIGN;
  const Range ins[9] = {
      strided_range(a.q, a.num_seqs, a.num_q_heads, a.q_seq_stride, a.q_head_stride, c.head_dim),
      range_of(c.codes[0], bytes[0]), range_of(c.scales[0], bytes[1]),
      range_of(c.codes[1], bytes[0]), range_of(c.scales[1], bytes[1]),
      range_of(a.page_table,
               a.num_seqs > 0 ? ((a.num_seqs - 1) * a.table_stride + a.max_pages) * 4 : 0),
      range_of(a.seq_lens, a.num_seqs * 4), range_of(c.global_scales[0], c.nvfp4 ? 4 : 0),
      range_of(c.global_scales[1], c.nvfp4 ? 4 : 0)};
  const int64_t heads = a.num_seqs * a.num_q_heads;
  const Range outs[4] = {range_of(a.out, heads * c.head_dim * 2),
                         range_of(a.lse, a.lse ? heads * 4 : 0),
                         range_of(a.workspace, work ? ws_bytes : 0),
                         range_of(a.status, a.status ? 4 : 0)};
  for (int i = 0; i < 4; ++i) {
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return MXFP4_EALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return MXFP4_EALIAS;
  }
  return from_cuda(mxfp4::launch_cache_attention(a, static_cast<cudaStream_t>(stream)));
}

int attention_call(const mxfp4::CacheArgs& c, const void* q, int64_t num_seqs, int32_t num_q_heads,
                   int64_t q_seq_stride, int64_t q_head_stride, const int32_t* page_table,
                   int64_t table_stride, int64_t max_pages, const int32_t* seq_lens,
                   float softmax_scale, int32_t window, void* workspace, size_t workspace_bytes,
                   void* out, float* lse, int32_t* status, void* stream) {
  mxfp4::AttentionArgs a{};
  a.cache = c;
  a.q = q;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.q_seq_stride = q_seq_stride;
  a.q_head_stride = q_head_stride;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.softmax_scale = softmax_scale;
  a.window = window;
  a.workspace = static_cast<float*>(workspace);
  a.out = out;
  a.lse = lse;
  a.status = status;
  return attention_checked(a, workspace_bytes, stream);
}

}  // namespace

extern "C" {

int mxfp4_matvec(const void* x, int64_t num_tokens, int64_t K, int64_t ldx, const uint8_t* codes,
                 const uint8_t* scales, int64_t N, void* y, int64_t ldy, int32_t y_f32,
                 void* stream) {
  return dense_matvec(x, num_tokens, K, ldx, codes, scales, nullptr, N, y, ldy, y_f32, false, false,
      stream);
}

int mxfp4_moe_matvec(const void* x, int64_t num_src_rows, int64_t K, int64_t ldx,
                     const int32_t* row_index, int64_t total_rows, const int32_t* expert_offsets,
                     int32_t E, const uint8_t* codes, const uint8_t* scales, int64_t N, void* y,
                     int64_t ldy, int32_t y_f32, int32_t* status, void* stream) {
  return moe_matvec(x, num_src_rows, K, ldx, row_index, total_rows, expert_offsets, E, codes,
      scales, nullptr, N, y, ldy, y_f32, status, false, false, stream);
}

int mxfp4_cache_write(const void* k, const void* v, int64_t num_tokens, int32_t num_heads,
                      int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                      int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                      int64_t num_pages, int32_t page_size, uint8_t* k_codes, uint8_t* k_scales,
                      uint8_t* v_codes, uint8_t* v_scales, int32_t* status, void* stream) {
  return write_checked(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr, num_pages,
      page_size, num_heads, head_dim, false, false), k, v, num_tokens, k_token_stride,
      k_head_stride, v_token_stride, v_head_stride, slots, status, stream);
}

int mxfp4_cache_read(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                     const uint8_t* v_scales, int64_t num_pages, int32_t page_size,
                     int32_t num_heads, int32_t head_dim, const int32_t* slots, int64_t num_tokens,
                     void* k_out, void* v_out, int32_t* status, void* stream) {
  return read_checked(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr, num_pages,
      page_size, num_heads, head_dim, false, false), slots, num_tokens, k_out, v_out, status,
      stream);
}

int mxfp4_cache_attention(const void* q, int64_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                          int64_t q_seq_stride, int64_t q_head_stride, const uint8_t* k_codes,
                          const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                          int64_t num_pages, int32_t page_size, int32_t num_kv_heads,
                          const int32_t* page_table, int64_t table_stride, int64_t max_pages,
                          const int32_t* seq_lens, float softmax_scale, int32_t window,
                          void* workspace, size_t workspace_bytes, void* out, float* lse,
                          int32_t* status, void* stream) {
  return attention_call(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr,
      num_pages, page_size, num_kv_heads, head_dim, false, false), q, num_seqs, num_q_heads,
      q_seq_stride, q_head_stride, page_table, table_stride, max_pages, seq_lens, softmax_scale,
      window, workspace, workspace_bytes, out, lse, status, stream);
}

int mxfp4_matvec_f16(const void* x, int64_t num_tokens, int64_t K, int64_t ldx,
                     const uint8_t* codes, const uint8_t* scales, int64_t N, void* y, int64_t ldy,
                     int32_t y_f32, void* stream) {
  return dense_matvec(x, num_tokens, K, ldx, codes, scales, nullptr, N, y, ldy, y_f32, true, false,
      stream);
}

int mxfp4_moe_matvec_f16(const void* x, int64_t num_src_rows, int64_t K, int64_t ldx,
                         const int32_t* row_index, int64_t total_rows,
                         const int32_t* expert_offsets, int32_t E, const uint8_t* codes,
                         const uint8_t* scales, int64_t N, void* y, int64_t ldy, int32_t y_f32,
                         int32_t* status, void* stream) {
  return moe_matvec(x, num_src_rows, K, ldx, row_index, total_rows, expert_offsets, E, codes,
      scales, nullptr, N, y, ldy, y_f32, status, true, false, stream);
}

int mxfp4_cache_write_f16(const void* k, const void* v, int64_t num_tokens, int32_t num_heads,
                          int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                          int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                          int64_t num_pages, int32_t page_size, uint8_t* k_codes, uint8_t* k_scales,
                          uint8_t* v_codes, uint8_t* v_scales, int32_t* status, void* stream) {
  return write_checked(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr, num_pages,
      page_size, num_heads, head_dim, true, false), k, v, num_tokens, k_token_stride, k_head_stride,
      v_token_stride, v_head_stride, slots, status, stream);
}

int mxfp4_cache_read_f16(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                         const uint8_t* v_scales, int64_t num_pages, int32_t page_size,
                         int32_t num_heads, int32_t head_dim, const int32_t* slots,
                         int64_t num_tokens, void* k_out, void* v_out, int32_t* status,
                         void* stream) {
  return read_checked(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr, num_pages,
      page_size, num_heads, head_dim, true, false), slots, num_tokens, k_out, v_out, status,
      stream);
}

int mxfp4_cache_attention_f16(const void* q, int64_t num_seqs, int32_t num_q_heads,
                              int32_t head_dim, int64_t q_seq_stride, int64_t q_head_stride,
                              const uint8_t* k_codes, const uint8_t* k_scales,
                              const uint8_t* v_codes, const uint8_t* v_scales, int64_t num_pages,
                              int32_t page_size, int32_t num_kv_heads, const int32_t* page_table,
                              int64_t table_stride, int64_t max_pages, const int32_t* seq_lens,
                              float softmax_scale, int32_t window, void* workspace,
                              size_t workspace_bytes, void* out, float* lse, int32_t* status,
                              void* stream) {
  return attention_call(cache_args(k_codes, k_scales, v_codes, v_scales, nullptr, nullptr,
      num_pages, page_size, num_kv_heads, head_dim, true, false), q, num_seqs, num_q_heads,
      q_seq_stride, q_head_stride, page_table, table_stride, max_pages, seq_lens, softmax_scale,
      window, workspace, workspace_bytes, out, lse, status, stream);
}

int mxfp4_matvec_nvfp4(const void* x, int64_t num_tokens, int64_t K, int64_t ldx,
                       const uint8_t* codes, const uint8_t* scales, const float* global_scale,
                       int64_t N, void* y, int64_t ldy, int32_t y_f32, void* stream) {
  return dense_matvec(x, num_tokens, K, ldx, codes, scales, global_scale, N, y, ldy, y_f32, false,
      true, stream);
}

int mxfp4_moe_matvec_nvfp4(const void* x, int64_t num_src_rows, int64_t K, int64_t ldx,
                           const int32_t* row_index, int64_t total_rows,
                           const int32_t* expert_offsets, int32_t E, const uint8_t* codes,
                           const uint8_t* scales, const float* global_scales, int64_t N, void* y,
                           int64_t ldy, int32_t y_f32, int32_t* status, void* stream) {
  return moe_matvec(x, num_src_rows, K, ldx, row_index, total_rows, expert_offsets, E, codes,
      scales, global_scales, N, y, ldy, y_f32, status, false, true, stream);
}

int mxfp4_cache_write_nvfp4(const void* k, const void* v, int64_t num_tokens, int32_t num_heads,
                            int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                            int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                            int64_t num_pages, int32_t page_size, const float* k_global,
                            const float* v_global, uint8_t* k_codes, uint8_t* k_scales,
                            uint8_t* v_codes, uint8_t* v_scales, int32_t* status, void* stream) {
  return write_checked(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_heads, head_dim, false, true), k, v, num_tokens, k_token_stride,
      k_head_stride, v_token_stride, v_head_stride, slots, status, stream);
}

int mxfp4_cache_read_nvfp4(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                           const uint8_t* v_scales, const float* k_global, const float* v_global,
                           int64_t num_pages, int32_t page_size, int32_t num_heads,
                           int32_t head_dim, const int32_t* slots, int64_t num_tokens, void* k_out,
                           void* v_out, int32_t* status, void* stream) {
  return read_checked(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_heads, head_dim, false, true), slots, num_tokens, k_out, v_out,
      status, stream);
}

int mxfp4_cache_attention_nvfp4(const void* q, int64_t num_seqs, int32_t num_q_heads,
                                int32_t head_dim, int64_t q_seq_stride, int64_t q_head_stride,
                                const uint8_t* k_codes, const uint8_t* k_scales,
                                const uint8_t* v_codes, const uint8_t* v_scales,
                                const float* k_global, const float* v_global, int64_t num_pages,
                                int32_t page_size, int32_t num_kv_heads, const int32_t* page_table,
                                int64_t table_stride, int64_t max_pages, const int32_t* seq_lens,
                                float softmax_scale, int32_t window, void* workspace,
                                size_t workspace_bytes, void* out, float* lse, int32_t* status,
                                void* stream) {
  return attention_call(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_kv_heads, head_dim, false, true), q, num_seqs, num_q_heads,
      q_seq_stride, q_head_stride, page_table, table_stride, max_pages, seq_lens, softmax_scale,
      window, workspace, workspace_bytes, out, lse, status, stream);
}

int mxfp4_matvec_nvfp4_f16(const void* x, int64_t num_tokens, int64_t K, int64_t ldx,
                           const uint8_t* codes, const uint8_t* scales, const float* global_scale,
                           int64_t N, void* y, int64_t ldy, int32_t y_f32, void* stream) {
  return dense_matvec(x, num_tokens, K, ldx, codes, scales, global_scale, N, y, ldy, y_f32, true,
      true, stream);
}

int mxfp4_moe_matvec_nvfp4_f16(const void* x, int64_t num_src_rows, int64_t K, int64_t ldx,
                               const int32_t* row_index, int64_t total_rows,
                               const int32_t* expert_offsets, int32_t E, const uint8_t* codes,
                               const uint8_t* scales, const float* global_scales, int64_t N,
                               void* y, int64_t ldy, int32_t y_f32, int32_t* status, void* stream) {
  return moe_matvec(x, num_src_rows, K, ldx, row_index, total_rows, expert_offsets, E, codes,
      scales, global_scales, N, y, ldy, y_f32, status, true, true, stream);
}

int mxfp4_cache_write_nvfp4_f16(const void* k, const void* v, int64_t num_tokens, int32_t num_heads,
                                int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                                int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                                int64_t num_pages, int32_t page_size, const float* k_global,
                                const float* v_global, uint8_t* k_codes, uint8_t* k_scales,
                                uint8_t* v_codes, uint8_t* v_scales, int32_t* status,
                                void* stream) {
  return write_checked(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_heads, head_dim, true, true), k, v, num_tokens, k_token_stride,
      k_head_stride, v_token_stride, v_head_stride, slots, status, stream);
}

int mxfp4_cache_read_nvfp4_f16(const uint8_t* k_codes, const uint8_t* k_scales,
                               const uint8_t* v_codes, const uint8_t* v_scales,
                               const float* k_global, const float* v_global, int64_t num_pages,
                               int32_t page_size, int32_t num_heads, int32_t head_dim,
                               const int32_t* slots, int64_t num_tokens, void* k_out, void* v_out,
                               int32_t* status, void* stream) {
  return read_checked(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_heads, head_dim, true, true), slots, num_tokens, k_out, v_out,
      status, stream);
}

int mxfp4_cache_attention_nvfp4_f16(const void* q, int64_t num_seqs, int32_t num_q_heads,
                                    int32_t head_dim, int64_t q_seq_stride, int64_t q_head_stride,
                                    const uint8_t* k_codes, const uint8_t* k_scales,
                                    const uint8_t* v_codes, const uint8_t* v_scales,
                                    const float* k_global, const float* v_global, int64_t num_pages,
                                    int32_t page_size, int32_t num_kv_heads,
                                    const int32_t* page_table, int64_t table_stride,
                                    int64_t max_pages, const int32_t* seq_lens, float softmax_scale,
                                    int32_t window, void* workspace, size_t workspace_bytes,
                                    void* out, float* lse, int32_t* status, void* stream) {
  return attention_call(cache_args(k_codes, k_scales, v_codes, v_scales, k_global, v_global,
      num_pages, page_size, num_kv_heads, head_dim, true, true), q, num_seqs, num_q_heads,
      q_seq_stride, q_head_stride, page_table, table_stride, max_pages, seq_lens, softmax_scale,
      window, workspace, workspace_bytes, out, lse, status, stream);
}

size_t mxfp4_cache_attention_workspace_bytes(int64_t num_seqs, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             int32_t page_size, int64_t max_pages) {
  if (num_seqs < 0 || num_q_heads < 0 || num_kv_heads < 1 || head_dim < 0 || page_size < 1 ||
      max_pages < 0)
    return 0;
  if (num_q_heads % num_kv_heads != 0 || head_dim % 32 != 0 ||
      head_dim > MXFP4_ATTENTION_MAX_HEAD_DIM || max_pages > INT32_MAX / page_size ||
      (num_q_heads > 0 && num_seqs > kMaxGrid / num_q_heads))
    return 0;
  return static_cast<size_t>(4 * mxfp4::attention_workspace_floats(
                                     num_seqs, num_q_heads, num_kv_heads, head_dim,
                                     max_pages * page_size));
}

}  // extern "C"

// attn_api.hip -- the C ABI of libfp8attn (declared in include/fp8attn.h):
// host-side argument validation, then the launches on the caller's stream.
// No allocation, no synchronisation, no exceptions across the boundary.
#include <limits.h>
#include <math.h>

#include "attn_launch.hpp"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // keeps every 64-bit offset in range
constexpr int64_t kMaxPage = ((int64_t)1 << 32) - 1;  // page strides: 32-bit factors of the kernels' offsets
constexpr int64_t kMaxTokens = ((int64_t)1 << 24) - 1;  // a launch holds below 2^32 threads of 256 a workgroup
constexpr int64_t kMaxRegions = (int64_t)1 << 22;        // below 2^32 threads of up to 512 a workgroup
constexpr int64_t kMaxHeads = 65536;

bool head_dim_ok(int64_t D) { return D >= 16 && D <= 256 && D % 16 == 0; }

// The sizes of a cache descriptor.
int cache_sizes(const fp8b_kv_cache* c) {
  if (!c) return FP8B_EINVAL;
  if (c->fmt != FP8B_FMT_E5M2 && c->fmt != FP8B_FMT_E4M3) return FP8B_EUNSUPPORTED;
  if (c->pages < 1 || c->pages > INT32_MAX || c->heads < 1 || c->heads > 1024 || !head_dim_ok(c->head_dim))
    return FP8B_EINVAL;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return FP8B_EINVAL;
  const int64_t rows = c->heads * c->page_size;
  if (c->page_stride < rows * c->head_dim || c->scale_page_stride < rows) return FP8B_EINVAL;
  if (c->page_stride > kMaxPage || c->scale_page_stride > kMaxPage) return FP8B_EINVAL;
  if (c->page_stride % 16 != 0 || c->scale_page_stride % 4 != 0) return FP8B_EALIGN;
  return FP8B_OK;
}

int cache_pointers(const fp8b_kv_cache* c) {
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return FP8B_EINVAL;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
    return FP8B_EALIGN;
  return FP8B_OK;
}

// bf16 rows [T][heads][D] with free strides.
int rows_check(const void* p, int64_t t, int64_t h) {
  if (!p) return FP8B_EINVAL;
  if (t < 0 || h < 0 || t > kMaxStride || h >= kMaxDim) return FP8B_EINVAL;
  if (!aligned(p, 16) || t % 8 != 0 || h % 8 != 0) return FP8B_EALIGN;
  return FP8B_OK;
}

int rope_check(const fp8b_rope* r, int64_t D) {
  if (!r) return FP8B_EINVAL;
  if (r->rot_dim < 0 || r->rot_dim > D || r->rot_dim % 16 != 0) return FP8B_EINVAL;
  if (!(r->eps >= 0.0f) || isinf(r->eps)) return FP8B_EINVAL;
  if (r->rot_dim > 0 && (!r->cos_sin || !r->positions || r->max_pos < 1 || r->max_pos > kMaxDim)) return FP8B_EINVAL;
  if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16) || !aligned(r->cos_sin, 16) || !aligned(r->positions, 8))
    return FP8B_EALIGN;
  return FP8B_OK;
}

fp8attn::Rows rows(const void* p, int64_t t, int64_t h, int64_t heads) {
  return {static_cast<const uint16_t*>(p), t, h, (int)heads};
}

// The arrays of a fused write.
struct QkvWrite {
  fp8attn::Rows q, k, v, q_out;
};
int qkv_write_check(const QkvWrite& w, const int64_t* slots, const fp8b_rope* rope, const fp8b_kv_cache* cache) {
  int rc = rope_check(rope, cache->head_dim);
  for (const fp8attn::Rows* r : {&w.q, &w.k, &w.v, &w.q_out})
    if (rc == FP8B_OK) rc = rows_check(r->p, r->t, r->h);
  if (rc == FP8B_OK) rc = cache_pointers(cache);
  if (rc != FP8B_OK) return rc;
  if (!slots) return FP8B_EINVAL;
  return aligned(slots, 8) ? FP8B_OK : FP8B_EALIGN;
}
int qkv_write(const QkvWrite& w, const int64_t* slots, int64_t T, const fp8b_rope* rope, const fp8b_kv_cache* cache,
              void* stream) {
  return fp8attn::launch_qkv(w.q, w.k, w.v, T, (int)cache->head_dim, rope, w.q_out, rows(nullptr, 0, 0, 0), slots,
                             cache, as_stream(stream));
}

int attention_sizes(const fp8b_kv_cache* c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                    int64_t window) {
  const int rc = cache_sizes(c);
  if (rc != FP8B_OK) return rc;
  if (B < 0 || B > kMaxDim || Hq < 1 || Hq > kMaxHeads || Hq % c->heads != 0) return FP8B_EINVAL;
  if (cols < 1 || cols > kMaxDim || max_context < 0 || max_context > kMaxDim || window < 0) return FP8B_EINVAL;
  const int64_t room = cols * c->page_size;
  const int64_t tokens = max_context < room ? max_context : room;
  const int64_t regions = B * c->heads * ((Hq / c->heads + 15) / 16);
  // (the pieces of a split launch may end up to 512 tiles past the last one)
  if (regions >= kMaxRegions || regions * (tokens / 32 + 1) > INT32_MAX - 1024) return FP8B_EINVAL;
  return FP8B_OK;
}

int attention_check(const fp8attn::Attention& a, const fp8b_kv_cache* c, int out_dtype) {
  if (out_dtype != FP8B_OUT_F32 && out_dtype != FP8B_OUT_BF16) return FP8B_EUNSUPPORTED;
  const int rc = attention_sizes(c, a.B, a.Hq, a.cols, a.max_context, a.window);
  if (rc != FP8B_OK) return rc;
  return isfinite(a.scale) && a.ld_table >= a.cols && a.ld_table <= kMaxStride ? FP8B_OK : FP8B_EINVAL;
}
int attention_pointers(const fp8attn::Attention& a, const fp8b_kv_cache* c) {
  int rc = rows_check(a.q, a.q_b, a.q_h);
  if (rc == FP8B_OK) rc = cache_pointers(c);
  if (rc != FP8B_OK) return rc;
  if (!a.table || !a.lens || !a.out) return FP8B_EINVAL;
  if (!aligned(a.table, 4) || !aligned(a.lens, 4) || !aligned(a.out, 16) || !aligned(a.lse, 4) ||
      !aligned(a.workspace, 16))
    return FP8B_EALIGN;
  const bool needed = fp8attn::attention_workspace(*c, a.B, a.Hq, a.cols, a.max_context, a.window) > 0;
  return a.workspace || !needed ? FP8B_OK : FP8B_EINVAL;
}

}  // namespace

#define FP8B_EXPORT __attribute__((visibility("default")))
#define FP8B_TRY(x)                  \
  do {                               \
    const int rc_ = (x);             \
    if (rc_ != FP8B_OK) return rc_;  \
  } while (0)

extern "C" {

FP8B_EXPORT int fp8b_attn_abi_version(void) { return FP8B_ATTN_ABI_VERSION; }

FP8B_EXPORT int fp8_qk_norm_rope(const void* q, int64_t q_t, int64_t q_h, const void* k, int64_t k_t, int64_t k_h,
                                 int64_t T, int64_t Hq, int64_t Hk, int64_t D, const fp8b_rope* rope, void* q_out,
                                 int64_t qo_t, int64_t qo_h, void* k_out, int64_t ko_t, int64_t ko_h, void* stream) {
  if (T < 0 || T > kMaxTokens || Hq < 0 || Hk < 0 || Hq > kMaxHeads || Hk > kMaxHeads || Hq + Hk < 1)
    return FP8B_EINVAL;
  if (!head_dim_ok(D)) return FP8B_EINVAL;
  if (T == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  FP8B_TRY(rope_check(rope, D));
  if (Hq > 0) FP8B_TRY(rows_check(q, q_t, q_h));
  if (Hk > 0) FP8B_TRY(rows_check(k, k_t, k_h));
  if (Hq > 0) FP8B_TRY(rows_check(q_out, qo_t, qo_h));
  if (Hk > 0) FP8B_TRY(rows_check(k_out, ko_t, ko_h));
  return fp8attn::launch_qkv(rows(q, q_t, q_h, Hq), rows(k, k_t, k_h, Hk), rows(nullptr, 0, 0, 0), T, (int)D, rope,
                             rows(q_out, qo_t, qo_h, Hq), rows(k_out, ko_t, ko_h, Hk), nullptr, nullptr,
                             as_stream(stream));
}

FP8B_EXPORT int fp8_kv_cache_write(const void* k, int64_t k_t, int64_t k_h, const void* v, int64_t v_t, int64_t v_h,
                                   const int64_t* slots, int64_t T, const fp8b_kv_cache* cache, void* stream) {
  FP8B_TRY(cache_sizes(cache));
  if (T < 0 || T > kMaxTokens) return FP8B_EINVAL;
  if (T == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  FP8B_TRY(rows_check(k, k_t, k_h));
  FP8B_TRY(rows_check(v, v_t, v_h));
  FP8B_TRY(cache_pointers(cache));
  if (!slots) return FP8B_EINVAL;
  if (!aligned(slots, 8)) return FP8B_EALIGN;
  return fp8attn::launch_qkv(rows(nullptr, 0, 0, 0), rows(k, k_t, k_h, cache->heads), rows(v, v_t, v_h, cache->heads),
                             T, (int)cache->head_dim, nullptr, rows(nullptr, 0, 0, 0), rows(nullptr, 0, 0, 0), slots,
                             cache, as_stream(stream));
}

FP8B_EXPORT int fp8_qkv_cache_write(const void* q, int64_t q_t, int64_t q_h, const void* k, int64_t k_t, int64_t k_h,
                                    const void* v, int64_t v_t, int64_t v_h, const int64_t* slots, int64_t T,
                                    int64_t Hq, const fp8b_rope* rope, const fp8b_kv_cache* cache, void* q_out,
                                    int64_t qo_t, int64_t qo_h, void* stream) {
  FP8B_TRY(cache_sizes(cache));
  if (T < 0 || T > kMaxTokens || Hq < 1 || Hq > kMaxHeads) return FP8B_EINVAL;
  if (T == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  const QkvWrite w = {rows(q, q_t, q_h, Hq), rows(k, k_t, k_h, cache->heads), rows(v, v_t, v_h, cache->heads),
                      rows(q_out, qo_t, qo_h, Hq)};
  FP8B_TRY(qkv_write_check(w, slots, rope, cache));
  return qkv_write(w, slots, T, rope, cache, stream);
}

FP8B_EXPORT int fp8_kv_cache_read(const fp8b_kv_cache* cache, const int32_t* table, int64_t ld_table, int64_t cols,
                                  const int32_t* offsets, int64_t B, int64_t R, void* k_out, void* v_out,
                                  void* stream) {
  FP8B_TRY(cache_sizes(cache));
  if (B < 1 || B > kMaxDim || cols < 1 || cols > kMaxDim || ld_table < cols || ld_table > kMaxStride)
    return FP8B_EINVAL;
  if (R < 0 || R > kMaxTokens) return FP8B_EINVAL;
  if (R == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  FP8B_TRY(cache_pointers(cache));
  if (!table || !offsets || !k_out || !v_out) return FP8B_EINVAL;
  if (!aligned(table, 4) || !aligned(offsets, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return FP8B_EALIGN;
  return fp8attn::launch_cache_read(*cache, table, ld_table, cols, offsets, B, R, static_cast<uint16_t*>(k_out),
                                    static_cast<uint16_t*>(v_out), as_stream(stream));
}

FP8B_EXPORT int64_t fp8_paged_attention_workspace(const fp8b_kv_cache* cache, int64_t B, int64_t Hq, int64_t cols,
                                                  int64_t max_context, int64_t window) {
  FP8B_TRY(attention_sizes(cache, B, Hq, cols, max_context, window));
  return fp8attn::attention_workspace(*cache, B, Hq, cols, max_context, window);
}

FP8B_EXPORT int fp8_paged_attention(const void* q, int64_t q_b, int64_t q_h, const fp8b_kv_cache* cache,
                                    const int32_t* table, int64_t ld_table, int64_t cols, const int32_t* lens,
                                    int64_t B, int64_t Hq, int64_t max_context, int64_t window, float scale, void* out,
                                    int out_dtype, float* lse, void* workspace, void* stream) {
  const fp8attn::Attention a = {static_cast<const uint16_t*>(q), q_b, q_h, table, ld_table, cols, lens, B, Hq,
                                max_context, window, scale, out, out_dtype == FP8B_OUT_F32, lse,
                                static_cast<float*>(workspace)};
  FP8B_TRY(attention_check(a, cache, out_dtype));
  if (B == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  FP8B_TRY(attention_pointers(a, cache));
  return fp8attn::launch_attention(*cache, a, as_stream(stream));
}

FP8B_EXPORT int fp8_attention_step(const void* q, int64_t q_b, int64_t q_h, const void* k, int64_t k_b, int64_t k_h,
                                   const void* v, int64_t v_b, int64_t v_h, const int64_t* slots, int64_t B,
                                   int64_t Hq, const fp8b_rope* rope, const fp8b_kv_cache* cache,
                                   const int32_t* table, int64_t ld_table, int64_t cols, const int32_t* lens,
                                   int64_t max_context, int64_t window, float scale, void* q_out, int64_t qo_b,
                                   int64_t qo_h, void* out, int out_dtype, float* lse, void* workspace, void* stream) {
  const fp8attn::Attention a = {static_cast<const uint16_t*>(q_out), qo_b, qo_h, table, ld_table, cols, lens, B, Hq,
                                max_context, window, scale, out, out_dtype == FP8B_OUT_F32, lse,
                                static_cast<float*>(workspace)};
  FP8B_TRY(attention_check(a, cache, out_dtype));
  if (B == 0) return FP8B_OK;  // nothing is read or written; empty arrays may be NULL
  const QkvWrite w = {rows(q, q_b, q_h, Hq), rows(k, k_b, k_h, cache->heads), rows(v, v_b, v_h, cache->heads),
                      rows(q_out, qo_b, qo_h, Hq)};
  FP8B_TRY(qkv_write_check(w, slots, rope, cache));
  FP8B_TRY(attention_pointers(a, cache));
  FP8B_TRY(qkv_write(w, slots, B, rope, cache, stream));
  return fp8attn::launch_attention(*cache, a, as_stream(stream));
}

}  // extern "C"

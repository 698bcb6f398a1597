// moe_api.hip -- the C ABI of libfp8moe (declared in include/fp8moe.h):
// host-side argument validation, then the launches on the caller's stream.
// No allocation, no synchronisation, no exceptions across the boundary.
#include <initializer_list>

#include "moe_launch.hpp"

namespace {

using fp8moe::Mat;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int64_t kMaxBytes = (int64_t)1 << 62;    // of an array, first row to last: offsets stay in 64 bits
constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxCols = (int64_t)1 << 29;    // of a row: 32-bit byte offsets, with room behind it
constexpr int64_t kMaxSlots = (int64_t)1 << 28;
constexpr int64_t kMaxK = 131071;                  // (2^17 - 1) products of at most 2^14 in 32 bits
constexpr int64_t kMaxN = (int64_t)1 << 25;
constexpr int64_t kMaxCodes = (int64_t)1 << 46;    // bytes of packed weights
constexpr int64_t kMaxOut = (int64_t)1 << 36;      // values of a product: launches of less than 2^32 threads
constexpr int64_t kMaxExpertRows = (int64_t)1 << 30;  // rows of all experts' weights, for the same

bool type_ok(int t) { return t == FP8B_OUT_F32 || t == FP8B_OUT_BF16; }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

Mat mat(const void* p, int type, int64_t ld) { return {const_cast<void*>(p), ld, type == FP8B_OUT_BF16}; }
// Whether rows `ld` items apart (which is no more than kMaxLd, and cols no less
// than 1) have offsets in range.
bool rows_fit(int64_t rows, int64_t ld, int64_t item) { return rows <= 1 || ld <= kMaxBytes / item / rows; }
int mat_check(const Mat& m, int64_t rows, int64_t cols) {
  if (!m.p || m.ld < cols || m.ld > kMaxLd || !rows_fit(rows, m.ld, m.bf16 ? 2 : 4)) return FP8B_EINVAL;
  return aligned(m.p, m.bf16 ? 2 : 4) ? FP8B_OK : FP8B_EALIGN;
}
// 4-byte arrays that have to be there.
int words_check(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return FP8B_EINVAL;
  for (const void* p : ps)
    if (!aligned(p, 4)) return FP8B_EALIGN;
  return FP8B_OK;
}

int sort_sizes(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || T >= kMaxTokens || E < 1 || E > 1024 || k < 1 || k > 64 || T * k >= kMaxSlots) return FP8B_EINVAL;
  return FP8B_OK;
}
int plan_check(const fp8moe::Plan& p, int64_t T, void* ws) {
  const int rc = words_check({p.offsets});
  if (rc != FP8B_OK || T == 0) return rc;
  const int rc2 = words_check({p.experts, p.row_index, p.token_rows});
  if (rc2 != FP8B_OK) return rc2;
  if (!ws && fp8moe::sort_blocks(T) > 1) return FP8B_EINVAL;
  return aligned(ws, 16) ? FP8B_OK : FP8B_EALIGN;
}

int row_sizes(int64_t T, int64_t N, int64_t k, int64_t R) {
  if (T < 0 || T >= kMaxTokens || N < 1 || N >= kMaxCols || k < 1 || k > 64 || R < 0 || R >= kMaxRows)
    return FP8B_EINVAL;
  return FP8B_OK;
}

int product_check(const fp8moe::Product& p, int64_t rows) {
  if (!p.a || !p.sa || !p.w || !p.sw || !p.y.p) return FP8B_EINVAL;
  if (p.lda < up(p.K, 128) || p.lda >= (1 << 24)) return FP8B_EINVAL;
  if (!aligned(p.a, 16) || p.lda % 16 != 0 || !aligned(p.w, 16) || !aligned(p.sa, 4) || !aligned(p.sw, 4) ||
      !aligned(p.bias, 4))
    return FP8B_EALIGN;
  return mat_check(p.y, rows, p.N);
}
int product_sizes(int64_t N, int64_t K, int out_dtype) {
  if (!type_ok(out_dtype)) return FP8B_EUNSUPPORTED;
  return N >= 1 && N <= kMaxN && K >= 1 && K <= kMaxK ? FP8B_OK : FP8B_EINVAL;
}

}  // namespace

#define FP8B_EXPORT __attribute__((visibility("default")))
#define FP8B_TRY(x)                 \
  do {                              \
    const int rc_ = (x);            \
    if (rc_ != FP8B_OK) return rc_; \
  } while (0)

extern "C" {

FP8B_EXPORT int fp8b_moe_abi_version(void) { return FP8B_MOE_ABI_VERSION; }

FP8B_EXPORT int64_t moe_sort_workspace(int64_t T, int64_t E, int64_t k) {
  FP8B_TRY(sort_sizes(T, E, k));
  const int64_t blocks = fp8moe::sort_blocks(T);
  return blocks > 1 ? blocks * up(E, 4) * (int64_t)sizeof(int32_t) : 0;
}

FP8B_EXPORT int moe_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k, int renormalize,
                          float* gates, int32_t* experts, int32_t* expert_offsets, int32_t* row_index,
                          int32_t* token_rows, void* workspace, void* stream) {
  if (!type_ok(dtype)) return FP8B_EUNSUPPORTED;
  FP8B_TRY(sort_sizes(T, E, k));
  if (k > E) return FP8B_EINVAL;
  const fp8moe::Plan p{experts, expert_offsets, row_index, token_rows};
  FP8B_TRY(plan_check(p, T, workspace));
  if (T > 0) {
    FP8B_TRY(mat_check(mat(logits, dtype, ld), T, E));
    FP8B_TRY(words_check({gates}));
  }
  return fp8moe::launch_route(mat(logits, dtype, ld), T, (int)E, (int)k, renormalize != 0, gates, p,
                              static_cast<int32_t*>(workspace), as_stream(stream));
}

FP8B_EXPORT int moe_sort(const int32_t* experts, int64_t T, int64_t E, int64_t k, int32_t* expert_offsets,
                         int32_t* row_index, int32_t* token_rows, void* workspace, void* stream) {
  FP8B_TRY(sort_sizes(T, E, k));
  const fp8moe::Plan p{const_cast<int32_t*>(experts), expert_offsets, row_index, token_rows};
  FP8B_TRY(plan_check(p, T, workspace));
  return fp8moe::launch_sort(T, (int)E, (int)k, p, static_cast<int32_t*>(workspace), as_stream(stream));
}

FP8B_EXPORT int moe_route_backward(const float* dgates, const void* logits, int dtype, int64_t ld, const float* gates,
                                   const int32_t* experts, int64_t T, int64_t E, int64_t k, int renormalize,
                                   void* dlogits, int64_t ld_d, void* stream) {
  if (!type_ok(dtype)) return FP8B_EUNSUPPORTED;
  FP8B_TRY(sort_sizes(T, E, k));
  if (T == 0) return FP8B_OK;
  if (!renormalize) FP8B_TRY(mat_check(mat(logits, dtype, ld), T, E));
  FP8B_TRY(words_check({dgates, gates, experts}));
  FP8B_TRY(mat_check(mat(dlogits, dtype, ld_d), T, E));
  return fp8moe::launch_route_backward(dgates, mat(logits, dtype, ld), gates, experts, T, (int)E, (int)k,
                                       renormalize != 0, mat(dlogits, dtype, ld_d), as_stream(stream));
}

FP8B_EXPORT int moe_gather(const void* x, int dtype, int64_t ld_x, int64_t T, int64_t N, const int32_t* token_rows,
                           int64_t k, int64_t R, void* rows, int64_t ld_r, void* stream) {
  if (!type_ok(dtype)) return FP8B_EUNSUPPORTED;
  FP8B_TRY(row_sizes(T, N, k, R));
  if (T == 0 || R == 0) return FP8B_OK;
  FP8B_TRY(mat_check(mat(x, dtype, ld_x), T, N));
  FP8B_TRY(words_check({token_rows}));
  FP8B_TRY(mat_check(mat(rows, dtype, ld_r), R, N));
  return fp8moe::launch_gather(mat(x, dtype, ld_x), T, N, token_rows, (int)k, R, mat(rows, dtype, ld_r),
                               as_stream(stream));
}

FP8B_EXPORT int moe_combine(const void* y, int y_dtype, int64_t ld_y, int64_t R, int64_t N, const int32_t* token_rows,
                            const float* gates, int64_t T, int64_t k, void* out, int out_dtype, int64_t ld_o,
                            void* stream) {
  if (!type_ok(y_dtype) || !type_ok(out_dtype)) return FP8B_EUNSUPPORTED;
  FP8B_TRY(row_sizes(T, N, k, R));
  if (T == 0) return FP8B_OK;
  if (R > 0) FP8B_TRY(mat_check(mat(y, y_dtype, ld_y), R, N));
  FP8B_TRY(words_check({token_rows}));
  if (!aligned(gates, 4)) return FP8B_EALIGN;
  FP8B_TRY(mat_check(mat(out, out_dtype, ld_o), T, N));
  return fp8moe::launch_combine(mat(y, y_dtype, ld_y), R, N, token_rows, gates, T, (int)k, mat(out, out_dtype, ld_o),
                                as_stream(stream));
}

FP8B_EXPORT int moe_combine_backward(const void* dout, int out_dtype, int64_t ld_o, const void* y, int y_dtype,
                                     int64_t ld_y, int64_t R, int64_t N, const int32_t* token_rows, const float* gates,
                                     int64_t T, int64_t k, void* dy, int64_t ld_dy, float* dgates, void* stream) {
  if (!type_ok(y_dtype) || !type_ok(out_dtype)) return FP8B_EUNSUPPORTED;
  FP8B_TRY(row_sizes(T, N, k, R));
  if (T == 0) return FP8B_OK;
  FP8B_TRY(mat_check(mat(dout, out_dtype, ld_o), T, N));
  if (R > 0) {
    FP8B_TRY(mat_check(mat(y, y_dtype, ld_y), R, N));
    FP8B_TRY(mat_check(mat(dy, y_dtype, ld_dy), R, N));
  }
  FP8B_TRY(words_check({token_rows, gates, dgates}));
  return fp8moe::launch_combine_backward(mat(dout, out_dtype, ld_o), mat(y, y_dtype, ld_y), R, N, token_rows, gates, T,
                                         (int)k, mat(dy, y_dtype, ld_dy), dgates, as_stream(stream));
}

FP8B_EXPORT int int8_quant(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x, int8_t* codes, int64_t ld_c,
                           float* scales, void* stream) {
  if (!type_ok(dtype)) return FP8B_EUNSUPPORTED;
  if (M < 0 || M >= kMaxTokens || K < 1 || K >= kMaxCols) return FP8B_EINVAL;
  if (M == 0) return FP8B_OK;
  FP8B_TRY(mat_check(mat(x, dtype, ld_x), M, K));
  if (!codes || ld_c < K || ld_c > kMaxLd || !rows_fit(M, ld_c, 1)) return FP8B_EINVAL;
  FP8B_TRY(words_check({scales}));
  return fp8moe::launch_quant(mat(x, dtype, ld_x), M, K, codes, ld_c, scales, as_stream(stream));
}

FP8B_EXPORT int int8_weight_pack(const int8_t* w, int64_t G, int64_t N, int64_t K, int64_t ld_w, int64_t stride_w,
                                 int8_t* w_packed, void* stream) {
  if (G < 1 || N < 1 || N > kMaxN || K < 1 || K > kMaxK) return FP8B_EINVAL;
  if (G >= kMaxCodes || up(N, 16) * up(K, 128) >= kMaxCodes / G) return FP8B_EINVAL;
  if (!w || !w_packed || ld_w < K || ld_w > kMaxLd || stride_w < 0 || stride_w > kMaxLd) return FP8B_EINVAL;
  if (!rows_fit(N, ld_w, 1) || !rows_fit(G, stride_w, 1)) return FP8B_EINVAL;
  if (!aligned(w_packed, 16)) return FP8B_EALIGN;
  return fp8moe::launch_pack(w, G, N, K, ld_w, stride_w, w_packed, as_stream(stream));
}

FP8B_EXPORT int int8_gemm(const int8_t* a, int64_t ld_a, const float* a_scales, const int8_t* w_packed,
                          const float* w_scales, const float* bias, int64_t M, int64_t N, int64_t K, void* y,
                          int64_t ld_y, int out_dtype, void* stream) {
  FP8B_TRY(product_sizes(N, K, out_dtype));
  if (M < 0 || M >= kMaxTokens || M * N > kMaxOut) return FP8B_EINVAL;
  if (M == 0) return FP8B_OK;
  const fp8moe::Product p{a, ld_a, a_scales, w_packed, w_scales, bias, N, K, mat(y, out_dtype, ld_y)};
  FP8B_TRY(product_check(p, M));
  return fp8moe::launch_gemm(p, M, as_stream(stream));
}

FP8B_EXPORT int int8_grouped_gemm(const int8_t* a, int64_t ld_a, const float* a_scales, int64_t T,
                                  const int32_t* row_index, const int32_t* expert_offsets, int64_t R, int64_t E,
                                  const int8_t* w_packed, const float* w_scales, int64_t N, int64_t K, void* y,
                                  int64_t ld_y, int out_dtype, void* stream) {
  FP8B_TRY(product_sizes(N, K, out_dtype));
  if (E < 1 || E > 1024 || R < 0 || R >= kMaxTokens || T < 1 || T >= kMaxTokens || (!row_index && T != R && R > 0))
    return FP8B_EINVAL;
  if (up(N, 16) * up(K, 128) >= kMaxCodes / E || R * N > kMaxOut || E * N > kMaxExpertRows) return FP8B_EINVAL;
  // the rows of a are reached by 32-bit offsets
  if (ld_a < 0 || ld_a >= (1 << 24) || T * ld_a >= (int64_t)1 << 32) return FP8B_EINVAL;
  if (R == 0) return FP8B_OK;
  const fp8moe::Product p{a, ld_a, a_scales, w_packed, w_scales, nullptr, N, K, mat(y, out_dtype, ld_y)};
  FP8B_TRY(product_check(p, R));
  FP8B_TRY(words_check({expert_offsets}));
  if (!aligned(row_index, 4)) return FP8B_EALIGN;
  return fp8moe::launch_grouped(p, T, row_index, expert_offsets, R, (int)E, as_stream(stream));
}

}  // extern "C"

/*
 * fp8attn.h -- C ABI of the attention side of a decode step on MI355X
 * (gfx950): libfp8attn.so, beside the linear layers of libfp8blk.so.
 *
 * Between the block GEMM that projects a token to queries, keys and values
 * and the one that projects the attention's output back, a serving step
 *   - norms each query and key head and rotates it by its position,
 *   - quantises the keys and values into a paged FP8 cache,
 *   - attends with one new token per sequence to that sequence's pages.
 *
 * Source of the cache format: "LLM 推理的 FP8 混合精度工程 2026", section 4
 * (FP8 KV cache, real-time amax), with the row quantiser of fp8_kv_quant and
 * fp8_act_quant (fp8blk.h), one scale per token and head.
 *
 * The conventions of fp8blk.h hold for every entry point here: device
 * pointers owned by the caller (the descriptor fp8b_kv_cache itself is a
 * host struct, read during the call only), a hipStream_t as void*,
 * asynchronous launches on that stream, validation on the host, fp8b_status
 * codes, no allocation, no synchronisation, thread-safe.  Every call may be
 * captured in a HIP graph: grids follow from the arguments' sizes, lengths
 * are read on the device.  "bf16" rows are read and written with 16-byte
 * accesses.  The device of the stream must be the one the pointers are on,
 * and with stream NULL it must be the current one.
 */
#ifndef FP8ATTN_H
#define FP8ATTN_H
#include <stdint.h>

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8B_ATTN_ABI_VERSION 1

/* Version of this ABI (FP8B_ATTN_ABI_VERSION). */
int fp8b_attn_abi_version(void);

/*
 * A paged key-value cache of one layer.  Page p, head h, place i (token i
 * of the page) holds
 *   codes   head_dim bytes at   codes + p * page_stride
 *                                     + (h * page_size + i) * head_dim
 *   scale   one float at        scales + p * scale_page_stride
 *                                     + h * page_size + i
 * for K and V alike; value = E5M2 or E4M3 value of the code times the scale.
 * Slot s is page s / page_size, place s % page_size.  A page's head is one
 * contiguous block, so an attention workgroup streams whole lines, and the
 * page strides let layers, or K and V, share one allocation.
 *
 *   k_codes, v_codes    16-byte aligned; k_scales, v_scales: 16-byte aligned.
 *                       Apart from one another, pages interlaced or not, in
 *                       a cache that is written.
 *   page_stride         bytes, >= heads * page_size * head_dim, a multiple
 *                       of 16, below 2^32; the same for K and V.
 *   scale_page_stride   floats, >= heads * page_size, a multiple of 4, below
 *                       2^32.
 *   pages      1 .. 2^31 - 1.
 *   page_size  tokens: 16, 32, 64, ... 4096 (a power of two).
 *   heads      1 .. 1024;  head_dim 16 .. 256, a multiple of 16.
 *   fmt        FP8B_FMT_E5M2 or FP8B_FMT_E4M3.
 */
typedef struct {
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int64_t page_stride, scale_page_stride;
  int64_t pages, page_size, heads, head_dim;
  int32_t fmt, reserved;
} fp8b_kv_cache;

/*
 * How queries and keys are normed and rotated (host struct).  Per head x of
 * D values, all in fp32:
 *   u[i] = x[i] / sqrt(mean_j x[j]^2 + eps) * weight[i]   (weight NULL: u = x)
 *   (the sum of squares has to be finite and the mean plus eps normal in fp32),
 *   for i < rot_dim / 2, with c = cos_sin[pos][i] and
 *   s = cos_sin[pos][rot_dim/2 + i]:
 *     (a, b) -> (a c - b s, b c + a s), where (a, b) is
 *     (u[i], u[i + rot_dim/2]), or (u[2i], u[2i + 1]) if interleaved;
 *   values from rot_dim on pass unrotated; then one rounding to bf16.
 *
 *   q_weight, k_weight  bf16 [D], 16-byte aligned, or NULL (no norm).
 *   eps        >= 0, finite (used with a weight only).
 *   cos_sin    float [max_pos][rot_dim], 16-byte aligned, contiguous, or
 *              NULL with rot_dim 0 (no rotation).
 *   positions  int64 [T] (8-byte aligned); values outside [0, max_pos) give
 *              unspecified rows but never fault.  NULL with rot_dim 0.
 *   rot_dim    0, or a multiple of 16 up to D.
 */
typedef struct {
  const void *q_weight, *k_weight;
  const float *cos_sin;
  const int64_t *positions;
  int64_t max_pos, rot_dim;
  float eps;
  int32_t interleaved;
} fp8b_rope;

/*
 * fp8_qk_norm_rope -- norm and rotate the queries and keys of T tokens.
 *
 *   q   bf16, token t's head h at q + t * q_t + h * q_h (strides in
 *       elements, multiples of 8, q_t <= 2^40, q_h < 2^30), 16-byte aligned;
 *       k likewise with Hk heads.
 *       Slices of a fused projection's output need no copy.
 *   q_out, k_out  bf16 with strides of their own, as q and k; rows apart from
 *       each other.  Either may be the very array it is computed from (the
 *       same address and strides) and may not overlap the inputs otherwise.
 *   T >= 0 (0 is a no-op), T < 2^24; Hq, Hk >= 0, not both 0, <= 65536
 *       (with 0 heads the pointers may be NULL); D 16 .. 256, % 16 == 0.
 */
int fp8_qk_norm_rope(const void *q, int64_t q_t, int64_t q_h, const void *k,
                     int64_t k_t, int64_t k_h, int64_t T, int64_t Hq,
                     int64_t Hk, int64_t D, const fp8b_rope *rope,
                     void *q_out, int64_t qo_t, int64_t qo_h, void *k_out,
                     int64_t ko_t, int64_t ko_h, void *stream);

/*
 * fp8_kv_cache_write -- quantise keys and values as they enter the cache:
 * per token and head, d = fp32(amax / Fmax) (1 if amax = 0; Fmax 57344 or
 * 448), codes = E(clamp(fp32(x / d), +-Fmax)), d to the scale.  A NaN in a
 * row becomes a NaN code and leaves the row's other values as they would be
 * without it; an infinity makes the scale NaN.
 *
 *   k, v    bf16, token t's head h at k + t * k_t + h * k_h (elements,
 *           multiples of 8), 16-byte aligned.
 *   slots   int64 [T] (8-byte aligned): where token t goes.  A slot outside
 *           [0, pages * page_size), such as -1 for padding, writes nothing.
 *           A slot named twice in a call holds either token's K and either
 *           token's V rows, whole or mixed; other slots are not affected.
 *   T       0 (a no-op) .. 2^24 - 1.
 */
int fp8_kv_cache_write(const void *k, int64_t k_t, int64_t k_h, const void *v,
                       int64_t v_t, int64_t v_h, const int64_t *slots,
                       int64_t T, const fp8b_kv_cache *cache, void *stream);

/*
 * fp8_qkv_cache_write -- the two calls above in one launch: queries normed
 * and rotated to q_out, keys normed, rotated, rounded to bf16 and quantised
 * into the cache, values quantised into the cache.  Bit-identical to
 * fp8_qk_norm_rope followed by fp8_kv_cache_write.  Queries of tokens whose
 * slot is outside the cache are written all the same.  q_out may be q itself
 * (the same address and strides) and may not overlap any input otherwise.
 */
int fp8_qkv_cache_write(const void *q, int64_t q_t, int64_t q_h,
                        const void *k, int64_t k_t, int64_t k_h,
                        const void *v, int64_t v_t, int64_t v_h,
                        const int64_t *slots, int64_t T, int64_t Hq,
                        const fp8b_rope *rope, const fp8b_kv_cache *cache,
                        void *q_out, int64_t qo_t, int64_t qo_h,
                        void *stream);

/*
 * fp8_kv_cache_read -- the cache back as bf16 rows, sequences one after the
 * other: row r of sequence b (offsets[b] <= r < offsets[b+1]) is its token
 * r - offsets[b], and out[r][h][i] = bf16_RNE(fp32(value(code) * scale)).
 *
 *   table    int32 [B][cols], rows ld_table apart: the pages of sequence b in
 *            order.  Page ids outside [0, pages), or a sequence longer than
 *            cols pages, give unspecified rows but never fault.
 *   offsets  int32 [B+1], non-decreasing, [0] = 0 (otherwise unspecified
 *            rows, no fault).  Rows from offsets[B] on are left as they were.
 *   R        rows of the outputs; 0 is a no-op.  R < 2^24.
 *   B, cols  >= 1, <= 2^30; ld_table >= cols.
 *   k_out, v_out  bf16 contiguous [R][heads][head_dim], 16-byte aligned,
 *            apart from each other and from the inputs.
 */
int fp8_kv_cache_read(const fp8b_kv_cache *cache, const int32_t *table,
                      int64_t ld_table, int64_t cols, const int32_t *offsets,
                      int64_t B, int64_t R, void *k_out, void *v_out,
                      void *stream);

/*
 * fp8_paged_attention -- attention of one new token per sequence over the
 * cache.  For sequence b of n = min(lens[b], max_context) tokens (n <= 0 is
 * none) and query head h, reading KV head h / (Hq / heads):
 *   seen  j in [max(0, n - window), n)      (window 0: all of [0, n))
 *   s_j = scale * sum_i q[b][h][i] * K[j][i]
 *   out[b][h] = sum_j e^(s_j - m) V[j] / sum_j e^(s_j - m),  m = max_j s_j
 *   lse[b][h] = m + ln(sum_j e^(s_j - m))
 * A row that sees nothing, or only scores of -inf, gives out 0 and lse -inf;
 * a NaN or +inf among the seen scores gives NaN.  A V code of a seen token
 * that is not finite makes its position of the KV head's rows NaN or
 * infinite, a V scale all their positions.  What lies in the pages
 * outside the seen range, NaN codes or scales included, has no effect.
 * Products and sums are fp32; the weights e^(s_j - m) enter the products
 * with V split into bf16 parts that keep at least 24 significant bits, as
 * long as the product of a weight and its V scale is at least 2^-100.  Sums are taken in a fixed order: the
 * same call gives the same bits.
 *
 *   q        bf16, row b's head h at q + b * q_b + h * q_h (elements,
 *            multiples of 8), 16-byte aligned.  It includes the new token
 *            only through lens: write its K and V first.
 *   table, ld_table, cols, B  as for fp8_kv_cache_read; B >= 0 (0 is a
 *            no-op).  All cols entries of a row have to be readable; entries
 *            beyond the seen tokens' pages may be read, and the pages they
 *            name loaded (ids are clamped), without effect on the results.
 *   lens     int32 [B].
 *   max_context  0 .. 2^30: lengths beyond it, or beyond cols * page_size, are
 *            cut to it; a tight value saves the splitting of short contexts.
 *   window   >= 0.
 *   Hq       a multiple of cache->heads, at most 65536.
 *   scale    finite.
 *   out      contiguous [B][Hq][head_dim], bf16 or fp32 (out_dtype), 16-byte
 *            aligned.  lse: float [B][Hq] or NULL.  Neither may overlap the
 *            inputs, the workspace or the other.
 *   workspace  fp8_paged_attention_workspace(...) bytes, 16-byte aligned;
 *            what it holds before the call does not matter.  Calls that may
 *            run at the same time need one each.  NULL where the size is 0.
 *   B * heads * ceil(Hq / heads / 16) < 2^22, and times (tokens / 32 + 1)
 *            < 2^31 - 1024, tokens being min(max_context, cols * page_size).
 *
 * fp8_paged_attention_workspace returns the bytes for these sizes (it
 * depends on sizes only), or a negative status for sizes that
 * fp8_paged_attention refuses.
 */
int64_t fp8_paged_attention_workspace(const fp8b_kv_cache *cache, int64_t B,
                                      int64_t Hq, int64_t cols,
                                      int64_t max_context, int64_t window);
int fp8_paged_attention(const void *q, int64_t q_b, int64_t q_h,
                        const fp8b_kv_cache *cache, const int32_t *table,
                        int64_t ld_table, int64_t cols, const int32_t *lens,
                        int64_t B, int64_t Hq, int64_t max_context,
                        int64_t window, float scale, void *out, int out_dtype,
                        float *lse, void *workspace, void *stream);

/*
 * fp8_attention_step -- the attention side of a decode step, B sequences with
 * one new token each: fp8_qkv_cache_write of the tokens (T = B), then
 * fp8_paged_attention of the queries in q_out; lens counts the new tokens.
 * Bit-identical to the two calls, with every argument checked before anything
 * is written.  The workspace is fp8_paged_attention's for the same sizes.
 */
int fp8_attention_step(const void *q, int64_t q_b, int64_t q_h, const void *k,
                       int64_t k_b, int64_t k_h, const void *v, int64_t v_b,
                       int64_t v_h, const int64_t *slots, int64_t B,
                       int64_t Hq, const fp8b_rope *rope,
                       const fp8b_kv_cache *cache, const int32_t *table,
                       int64_t ld_table, int64_t cols, const int32_t *lens,
                       int64_t max_context, int64_t window, float scale,
                       void *q_out, int64_t qo_b, int64_t qo_h, void *out,
                       int out_dtype, float *lse, void *workspace,
                       void *stream);

#ifdef __cplusplus
}
#endif
#endif

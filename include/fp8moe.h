/*
 * fp8moe.h -- C ABI of expert routing and of the W8A8 layers in 8-bit
 * integers on MI355X (gfx950): libfp8moe.so, beside the FP8 linear layers of
 * libfp8blk.so.
 *
 * A mixture-of-experts layer picks k of E experts for each token, sorts the
 * (token, slot) pairs by expert, runs each expert's product on its rows and
 * sums the weighted rows back to their tokens.  fp8_grouped_gemm (fp8blk.h)
 * and int8_grouped_gemm take the plan that moe_route or moe_sort make;
 * moe_combine takes their rows.  The integer layers are the W8A8 form with
 * one scale per token and one per output channel; the products are summed in
 * 32-bit integers, exactly.
 *
 * Sources: the DeepSeek-V3 guide's configuration table (256 routed experts, 8
 * active per token) and the INT8 rows of the quantisation tables of "量化: FP8
 * 与混合精度推理" and of the "FP8 推理" notes (per-token activations, per-channel
 * weights).  Row order (expert, token, slot) is the one of fp8_grouped_gemm.
 *
 * The conventions of fp8blk.h hold for every entry point here: device
 * pointers owned by the caller, a hipStream_t as void*, asynchronous launches
 * on that stream, validation on the host, fp8b_status codes, no allocation,
 * no synchronisation, thread-safe, no global state.  Every call may be
 * captured in a HIP graph: grids follow from the arguments' sizes, plans are
 * read on the device.  The device of the stream must be the one the pointers
 * are on, and with stream NULL it must be the current one.  Outputs share no
 * memory with each other or with inputs.
 *
 * Types of arrays that may be fp32 or bf16 are given by fp8b_out_dtype.
 * Leading dimensions ld_* are in elements, at least the row length, at most
 * 2^40, and rows times ld_* times the element's size at most 2^62 bytes where
 * there is more than one row; arrays need the alignment of their type only,
 * unless stated.
 */
#ifndef FP8MOE_H
#define FP8MOE_H
#include <stdint.h>

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8B_MOE_ABI_VERSION 1

/* Version of this ABI (FP8B_MOE_ABI_VERSION). */
int fp8b_moe_abi_version(void);

/*
 * The plan of T tokens with k slots each, R = T * k rows:
 *   experts         int32 [T][k]  expert of (token, slot), -1 for none
 *   expert_offsets  int32 [E+1]   rows of expert e: [e] <= r < [e+1]; [0] = 0;
 *                                 [E] = rows in use (R less the empty slots)
 *   row_index       int32 [R]     token of row r; -1 from row [E] on
 *   token_rows      int32 [T][k]  row of (token, slot), -1 for none
 * with rows in the order of (expert, token, slot).
 *   T >= 0, T < 2^24;  1 <= E <= 1024;  1 <= k <= 64, k <= E for moe_route;
 *   T * k < 2^28.
 */

/* Bytes of workspace that moe_route and moe_sort need for T tokens (may be
 * 0), or a negative status.  Its contents before and after a call mean
 * nothing; calls that may run at the same time need one each. */
int64_t moe_sort_workspace(int64_t T, int64_t E, int64_t k);

/*
 * moe_route -- choose each token's experts and make the plan.
 *   Slot j's expert is the one with the j-th largest logit of the token, the
 *   lower id first among equal ones (-0 equals 0).  A logit of -inf is never
 *   chosen: slots without an expert have experts -1, gates 0, token_rows -1.
 *   A NaN counts as larger than any number.
 *   gates[t][j] = exp(l[e_j] - m) / sum exp(l[e] - m), the sum over the
 *   token's chosen experts (renormalize) or over all E (otherwise), in fp32;
 *   a NaN or +inf among the logits summed over makes the token's gates NaN.
 *
 *   logits     fp32 or bf16 [T][ld].
 *   gates      float [T][k];  the plan as above;  workspace 16-byte aligned.
 *   T = 0 writes expert_offsets (zeros) alone.  A token's gates have the same
 *   bits in a batch of any size.
 */
int moe_route(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E,
              int64_t k, int renormalize, float *gates, int32_t *experts,
              int32_t *expert_offsets, int32_t *row_index, int32_t *token_rows,
              void *workspace, void *stream);

/*
 * moe_sort -- the plan alone, for experts chosen elsewhere: ids outside
 * [0, E) count as -1.  A token may name an expert more than once.
 */
int moe_sort(const int32_t *experts, int64_t T, int64_t E, int64_t k,
             int32_t *expert_offsets, int32_t *row_index, int32_t *token_rows,
             void *workspace, void *stream);

/*
 * moe_route_backward -- the gradient of the gates with respect to the
 * logits.  With D = sum_j gates[t][j] * dgates[t][j] over the token's slots
 * that have an expert:
 *   renormalize: dlogits[t][e_j] = gates[t][j] * (dgates[t][j] - D), 0 for
 *     experts that were not chosen (the logits are not read);
 *   otherwise, with p = softmax(logits[t]): dlogits[t][e] =
 *     (gates[t][j] * dgates[t][j] if e = e_j) - p[e] * D.
 *   An expert named by several slots gets the sum.  A token without experts
 *   gets zeros; dgates of empty slots are not looked at.
 *
 *   logits   as in moe_route (NULL with renormalize);
 *   dlogits  of the same type, [T][ld_d].
 */
int moe_route_backward(const float *dgates, const void *logits, int dtype,
                       int64_t ld, const float *gates, const int32_t *experts,
                       int64_t T, int64_t E, int64_t k, int renormalize,
                       void *dlogits, int64_t ld_d, void *stream);

/*
 * moe_gather -- token rows to their experts:
 *   rows[token_rows[t][j]] = x[t].
 *   Rows that no slot names are left as they were.
 *
 *   x [T][ld_x], rows [R][ld_r], both of `dtype`;  N >= 1 columns, < 2^29;
 *   token_rows outside [0, R) count as -1 (no row); no row is named twice.
 *   T < 2^24; 0 <= R < 2^30; 1 <= k <= 64.
 */
int moe_gather(const void *x, int dtype, int64_t ld_x, int64_t T, int64_t N,
               const int32_t *token_rows, int64_t k, int64_t R, void *rows,
               int64_t ld_r, void *stream);

/*
 * moe_combine -- rows back to their tokens:
 *   out[t][n] = sum_j gates[t][j] * y[token_rows[t][j]][n]
 *   over the slots that have a row, in fp32 in slot order (one fused
 *   multiply-add each), rounded once; gates NULL counts as ones (the
 *   gradient of moe_gather).  Rows and gates of empty slots are not read.
 *
 *   y [R][ld_y] of y_dtype, out [T][ld_o] of out_dtype; the rest as above.
 */
int moe_combine(const void *y, int y_dtype, int64_t ld_y, int64_t R, int64_t N,
                const int32_t *token_rows, const float *gates, int64_t T,
                int64_t k, void *out, int out_dtype, int64_t ld_o,
                void *stream);

/*
 * moe_combine_backward -- the gradients of moe_combine:
 *   dy[token_rows[t][j]][n] = gates[t][j] * dout[t][n]   (rounded once),
 *   dgates[t][j] = sum_n dout[t][n] * y[token_rows[t][j]][n]   (in fp32;
 *   0 for an empty slot).
 *   Rows of dy that no slot names are left as they were.
 *
 *   dout [T][ld_o] of out_dtype; y [R][ld_y] and dy [R][ld_dy] of y_dtype.
 */
int moe_combine_backward(const void *dout, int out_dtype, int64_t ld_o,
                         const void *y, int y_dtype, int64_t ld_y, int64_t R,
                         int64_t N, const int32_t *token_rows,
                         const float *gates, int64_t T, int64_t k, void *dy,
                         int64_t ld_dy, float *dgates, void *stream);

/*
 * int8_quant -- one scale per row (a token's activations, an output channel's
 * weights):
 *   amax = max |x[m][k]|, d = fp32(amax / 127), at least 2^-126 and 1 if
 *   amax = 0; codes[m][k] = the whole number nearest to fp32(x[m][k] / d),
 *   ties to even, from -127 to 127; scales[m] = d.
 *   A row that holds a NaN has scale NaN, one that holds an infinity and no
 *   NaN has scale +inf; both have codes 0, so what is computed from them is
 *   NaN.
 *
 *   x       fp32 or bf16 [M][ld_x].
 *   codes   int8 [M][ld_c];  scales float [M].
 *   M >= 0 (0 is a no-op), < 2^24; K >= 1, < 2^29.
 */
int int8_quant(const void *x, int dtype, int64_t M, int64_t K, int64_t ld_x,
               int8_t *codes, int64_t ld_c, float *scales, void *stream);

/*
 * int8_weight_pack -- weight codes into the layout that the products read:
 * the chunks of fp8_weight_pack (fp8blk.h), the matrix filled up with zeros
 * to a multiple of 16 rows and of 128 columns.  With Np = N rounded up to
 * 16 and Kp = K rounded up to 128, one [N][K] matrix takes Np * Kp bytes:
 * chunk (kc, p), kc < Kp/64, p < Np/16, at byte (kc * Np/16 + p) * 1024;
 * byte 256*g + 16*r + b of it is the code of row 16p + r, column
 * 64kc + 16g + b.
 *
 *   w         int8, matrix i, row n at w + i * stride_w + n * ld_w
 *             (0 <= stride_w <= 2^40).
 *   G >= 1; 1 <= N <= 2^25; 1 <= K <= 131071; G * Np * Kp < 2^46;
 *   G * stride_w <= 2^62.
 *   w_packed  G * Np * Kp bytes, 16-byte aligned, not overlapping w.
 */
int int8_weight_pack(const int8_t *w, int64_t G, int64_t N, int64_t K,
                     int64_t ld_w, int64_t stride_w, int8_t *w_packed,
                     void *stream);

/*
 * int8_gemm -- y[m][n] = fp32(sum_k a[m][k] * w[n][k]) * a_scales[m] *
 * w_scales[n] + bias[n], the sum in 32-bit integers (exact: K <= 131071
 * products of at most 2^14), the rest in fp32, rounded once to y's type.  The
 * product of the two scales alone may leave fp32's range; a scale of 0 gives 0
 * beside any number.
 *
 *   a         int8 [M][ld_a], 16-byte aligned, ld_a % 16 == 0, ld_a >= Kp (K
 *             rounded up to 128): the bytes from K to Kp of every row are
 *             read, and do not count.
 *   a_scales  float [M];  w_scales float [N];  bias float [N] or NULL.
 *   w_packed  from int8_weight_pack, 16-byte aligned.
 *   M >= 0 (0 is a no-op), < 2^24; 1 <= N <= 2^25; M * N <= 2^36;
 *   1 <= K <= 131071; ld_a < 2^24.
 *   y         [M][ld_y] of out_dtype.
 */
int int8_gemm(const int8_t *a, int64_t ld_a, const float *a_scales,
              const int8_t *w_packed, const float *w_scales, const float *bias,
              int64_t M, int64_t N, int64_t K, void *y, int64_t ld_y,
              int out_dtype, void *stream);

/*
 * int8_grouped_gemm -- int8_gemm per expert, the gather inside: row r of
 * expert e (expert_offsets[e] <= r < expert_offsets[e+1]) is row
 * t = row_index[r] of a, or row r itself where row_index is NULL (a in
 * expert order, T = R):
 *   y[r][n] = fp32(sum_k a[t][k] * w[e][n][k]) * a_scales[t] * w_scales[e][n]
 *   Rows from expert_offsets[E] on are left as they were.
 *
 *   expert_offsets  int32 [E+1], non-decreasing within 0 .. R; others, or
 *                   tokens outside [0, T), give unspecified rows of y but
 *                   never fault.
 *   T >= 1, T * ld_a < 2^32 (rows are gathered with 32-bit offsets);
 *   0 <= R < 2^24 (0 is a no-op); 1 <= E <= 1024; R * N <= 2^36; E * N <= 2^30.
 *   w_packed  of E matrices;  w_scales float [E][N].
 */
int int8_grouped_gemm(const int8_t *a, int64_t ld_a, const float *a_scales,
                      int64_t T, const int32_t *row_index,
                      const int32_t *expert_offsets, int64_t R, int64_t E,
                      const int8_t *w_packed, const float *w_scales, int64_t N,
                      int64_t K, void *y, int64_t ld_y, int out_dtype,
                      void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8MOE_H */

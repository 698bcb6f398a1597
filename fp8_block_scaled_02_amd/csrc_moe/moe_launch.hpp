// moe_launch.hpp -- host-side launch plumbing of libfp8moe.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8moe.h"

namespace fp8moe {

inline int check_launch() {
  return hipGetLastError() == hipSuccess ? FP8B_OK : FP8B_ELAUNCH;
}

// A 2-D array of fp32 or bf16 with a leading dimension in elements.
struct Mat {
  void* p;
  int64_t ld;
  bool bf16;
};

// The plan's arrays.
struct Plan {
  int32_t *experts, *offsets, *row_index, *token_rows;
};

// Workgroups of a sort that count apart; each takes E words of workspace, rounded up to 4 (1: none needed).
int64_t sort_blocks(int64_t T);
int launch_route(const Mat& logits, int64_t T, int E, int k, bool renormalize, float* gates, const Plan& p, int32_t* ws,
                 hipStream_t s);
// p.experts is read
int launch_sort(int64_t T, int E, int k, const Plan& p, int32_t* ws, hipStream_t s);
int launch_route_backward(const float* dgates, const Mat& logits, const float* gates, const int32_t* experts, int64_t T,
                          int E, int k, bool renormalize, const Mat& dlogits, hipStream_t s);

int launch_gather(const Mat& x, int64_t T, int64_t N, const int32_t* token_rows, int k, int64_t R, const Mat& rows,
                  hipStream_t s);
int launch_combine(const Mat& y, int64_t R, int64_t N, const int32_t* token_rows, const float* gates, int64_t T, int k,
                   const Mat& out, hipStream_t s);
int launch_combine_backward(const Mat& dout, const Mat& y, int64_t R, int64_t N, const int32_t* token_rows,
                            const float* gates, int64_t T, int k, const Mat& dy, float* dgates, hipStream_t s);

int launch_quant(const Mat& x, int64_t M, int64_t K, int8_t* codes, int64_t ld_c, float* scales, hipStream_t s);
int launch_pack(const int8_t* w, int64_t G, int64_t N, int64_t K, int64_t ld, int64_t stride, int8_t* out,
                hipStream_t s);

// The products: a [.][lda] codes, packed weights, y [.][y.ld].
struct Product {
  const int8_t* a;
  int64_t lda;
  const float* sa;
  const int8_t* w;
  const float *sw, *bias;
  int64_t N, K;
  Mat y;
};
int launch_gemm(const Product& p, int64_t M, hipStream_t s);
int launch_grouped(const Product& p, int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, int E,
                   hipStream_t s);

}  // namespace fp8moe

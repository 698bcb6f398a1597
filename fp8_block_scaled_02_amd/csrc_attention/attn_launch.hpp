// attn_launch.hpp -- host-side launch plumbing of libfp8attn.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8attn.h"

namespace fp8attn {

inline int check_launch() {
  return hipGetLastError() == hipSuccess ? FP8B_OK : FP8B_ELAUNCH;
}

// [T][heads][D] bf16 with free token and head strides (elements).
struct Rows {
  const uint16_t* p;
  int64_t t, h;
  int heads;
};

// q: Hq rows per token or none; k, v: cache->heads rows or none.  With a
// cache, k and v go to their slots, otherwise k goes to k_out.
int launch_qkv(const Rows& q, const Rows& k, const Rows& v, int64_t T, int D, const fp8b_rope* rope, const Rows& q_out,
               const Rows& k_out, const int64_t* slots, const fp8b_kv_cache* cache, hipStream_t s);
int launch_cache_read(const fp8b_kv_cache& c, const int32_t* table, int64_t ld_table, int64_t cols,
                      const int32_t* offsets, int64_t B, int64_t R, uint16_t* k_out, uint16_t* v_out, hipStream_t s);

struct Attention {
  const uint16_t* q;
  int64_t q_b, q_h;
  const int32_t* table;
  int64_t ld_table, cols;
  const int32_t* lens;
  int64_t B, Hq, max_context, window;
  float scale;
  void* out;
  int out_f32;
  float* lse;
  float* workspace;
};
int64_t attention_workspace(const fp8b_kv_cache& c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                            int64_t window);
int launch_attention(const fp8b_kv_cache& c, const Attention& a, hipStream_t s);

}  // namespace fp8attn

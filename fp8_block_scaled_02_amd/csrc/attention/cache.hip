// cache.hip -- what surrounds the attention kernel on a paged FP8 cache
// (layout: fp8b_kv_cache in include/fp8attn.h): query/key norms with the
// position rotation, the quantising write, and reading back.
#include "../common.hpp"
#include "attn_launch.hpp"

namespace fp8attn {

using namespace fp8blk;

// ---- norm, rotate, quantise ------------------------------------------------

struct QkvArgs {
  Rows q, k, v;
  int64_t T;
  int D;
  const uint16_t *q_weight, *k_weight;
  const float* cos_sin;
  const int64_t* positions;
  int64_t max_pos;
  int rot;
  float eps;
  Rows q_out, k_out;
  const int64_t* slots;
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int64_t page_stride, scale_page_stride, total_slots;
  int page_shift, cache_heads;
  int slot_shift;  // log2 of the row slots of a workgroup that one token takes
  int items, token_items;  // rows of a slot; token_items > 1: they are of that many tokens
};

// Sum and maximum over the LPR (8, 16 or 32) adjacent lanes of a row: quad
// swaps, half-row mirror, row mirror, then the neighbouring row of 16.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
  if (LPR >= 16) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));
  if (LPR >= 32) v += __shfl_xor(v, 16);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max_nonneg(float v) {
  uint32_t u = __float_as_uint(v);
  u = umax_dpp<0xB1>(u);
  u = umax_dpp<0x4E>(u);
  u = umax_dpp<0x141>(u);
  if (LPR >= 16) u = umax_dpp<0x140>(u);
  if (LPR >= 32) {
    const uint32_t o = (uint32_t)__shfl_xor((int)u, 16);
    u = o > u ? o : u;
  }
  return __uint_as_float(u);
}

__device__ __forceinline__ void unpack8(const u32x4& w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2 b = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
    o[i] = __builtin_bit_cast(uint32_t, b);
  }
  return o;
}

// One row (token, head) per LPR lanes, 8 values per lane, LPR * 8 >= D; the
// lanes past D hold zeros.  A workgroup's 256 / LPR row slots are split into
// groups of 2^slot_shift that share a token; rows are numbered queries, keys,
// values.  A slot takes `items` rows, the next one loaded while this one is
// worked on: other heads of its token, whose cos and sin it keeps, or
// (nothing to rotate, heads no more than slots) the same head of later tokens.
//
// FMT: 0 no cache (keys to k_out), 1 E5M2, 2 E4M3.  ROPE: 0 none, 1 halves,
// 2 interleaved.  HBM-bound: 2 bytes in and 2 (or 1 and a scale) out per
// value; the arithmetic is ~10 operations per value.
template <int LPR, int ROPE, int FMT>
__global__ __launch_bounds__(256) void qkv_kernel(const QkvArgs a) {
  constexpr int kSlots = 256 / LPR;
  const int lane = threadIdx.x & (LPR - 1);
  const int slot = threadIdx.x / LPR;
  const int per_token = 1 << a.slot_shift;
  const int tokens = kSlots >> a.slot_shift;  // of a workgroup at a time
  const int rows = a.q.heads + a.k.heads + a.v.heads;
  int64_t t = (int64_t)blockIdx.x * tokens * a.token_items + (slot >> a.slot_shift);
  int r = (int)blockIdx.y * per_token + (slot & (per_token - 1));
  const int row_step = (int)gridDim.y * per_token;
  if (t >= a.T || r >= rows) return;
  const int e0 = 8 * lane;
  const bool on = e0 < a.D;
  const int half = a.rot >> 1;

  auto load = [&](int64_t tt, int rr) {
    const bool is_q = rr < a.q.heads, is_k = !is_q && rr < a.q.heads + a.k.heads;
    const Rows& src = is_q ? a.q : (is_k ? a.k : a.v);
    const int h = rr - (is_q ? 0 : (is_k ? a.q.heads : a.q.heads + a.k.heads));
    u32x4 x = {0, 0, 0, 0};
    if (on)
      x = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(src.p + tt * src.t + (int64_t)h * src.h + e0));
    return x;
  };
  u32x4 next = load(t, r);
  int64_t next_slot = FMT != 0 ? a.slots[t] : 0;

  float cs[8], sn[8];
  int partner = lane;
  if (ROPE != 0) {
    int64_t pos = a.positions[t];
    pos = pos < 0 ? 0 : (pos >= a.max_pos ? a.max_pos - 1 : pos);
    const float* tab = a.cos_sin + pos * a.rot;
    if (ROPE == 1) {
      const int i0 = e0 < half ? e0 : e0 - half;
      if (e0 < a.rot) {
        partner = e0 < half ? lane + (half >> 3) : lane - (half >> 3);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cs[i] = tab[i0 + i];
          // the first of a pair gets a c - b s, the second b c + a s
          sn[i] = e0 < half ? -tab[half + i0 + i] : tab[half + i0 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = e0 < a.rot ? tab[(e0 >> 1) + i] : 1.0f;
        sn[i] = e0 < a.rot ? tab[half + (e0 >> 1) + i] : 0.0f;
      }
    }
  }

  for (int left = a.items; left > 0; --left) {
    u32x4 raw = next;
    const int64_t sl = next_slot, tt = t;
    const int rr = r;
    if (a.token_items > 1) t += tokens;
    else r += row_step;
    const bool last = left == 1 || t >= a.T || r >= rows;
    if (!last) {
      next = load(t, r);
      if (FMT != 0 && a.token_items > 1) next_slot = a.slots[t];
    }
    const int kind = rr < a.q.heads ? 0 : (rr < a.q.heads + a.k.heads ? 1 : 2);
    const int h = kind == 0 ? rr : (kind == 1 ? rr - a.q.heads : rr - a.q.heads - a.k.heads);
    float f[8];
    if (FMT == 0 || kind < 2) {
      unpack8(raw, f);
      const uint16_t* w = kind == 0 ? a.q_weight : a.k_weight;
      if (w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
        ss = row_sum<LPR>(ss);
        const float rn = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        u32x4 wr = {0, 0, 0, 0};
        if (on) wr = *reinterpret_cast<const u32x4*>(w + e0);
        float wf[8];
        unpack8(wr, wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * rn * wf[i];
      }
      if (ROPE == 1) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl(f[i], partner, LPR);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = e0 < a.rot ? __builtin_fmaf(f[i], cs[i], o[i] * sn[i]) : f[i];
      } else if (ROPE == 2) {
        if (e0 < a.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = f[2 * i], y = f[2 * i + 1];
            f[2 * i] = __builtin_fmaf(x, cs[i], -(y * sn[i]));
            f[2 * i + 1] = __builtin_fmaf(y, cs[i], x * sn[i]);
          }
        }
      }
      raw = pack8(f);  // one rounding to bf16
    }
    if (FMT == 0 || kind == 0) {
      const Rows& dst = kind == 0 ? a.q_out : a.k_out;
      uint16_t* dp = const_cast<uint16_t*>(dst.p) + tt * dst.t + (int64_t)h * dst.h + e0;
      if (on) *reinterpret_cast<u32x4*>(dp) = raw;
    } else if (sl >= 0 && sl < a.total_slots) {
      constexpr float kMax = FMT == 1 ? 57344.0f : 448.0f;
      unpack8(raw, f);
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
      amax = row_max_nonneg<LPR>(amax);
      const float d = block_scale(amax, kMax, 1.0f / kMax);
      const BlockDivisor bd = make_divisor(amax, d);
      float v[8];
      divide_block(f, v, bd);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -kMax), kMax);
      u32x2 codes;
      codes[0] = FMT == 1 ? pack4_e5m2(v[0], v[1], v[2], v[3]) : pack4_e4m3(v[0], v[1], v[2], v[3]);
      codes[1] = FMT == 1 ? pack4_e5m2(v[4], v[5], v[6], v[7]) : pack4_e4m3(v[4], v[5], v[6], v[7]);
      const int64_t page = sl >> a.page_shift;
      const int64_t in_page = ((int64_t)h << a.page_shift) + (sl & ((1 << a.page_shift) - 1));
      uint8_t* cp = (kind == 1 ? a.k_codes : a.v_codes) + page * a.page_stride;
      float* sp = (kind == 1 ? a.k_scales : a.v_scales) + page * a.scale_page_stride;
      if (on) *reinterpret_cast<u32x2*>(cp + in_page * a.D + e0) = codes;
      if (lane == 0) sp[in_page] = d;
    }
    if (last) return;
  }
}

constexpr int kManyWgs = 1024;
constexpr int kTokenItems = 4;

int launch_qkv(const Rows& q, const Rows& k, const Rows& v, int64_t T, int D, const fp8b_rope* rope, const Rows& q_out,
               const Rows& k_out, const int64_t* slots, const fp8b_kv_cache* cache, hipStream_t s) {
  QkvArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.T = T;
  a.D = D;
  int kind = 0;
  if (rope) {
    a.q_weight = static_cast<const uint16_t*>(rope->q_weight);
    a.k_weight = static_cast<const uint16_t*>(rope->k_weight);
    a.eps = rope->eps;
    if (rope->rot_dim > 0) {
      a.cos_sin = rope->cos_sin;
      a.positions = rope->positions;
      a.max_pos = rope->max_pos;
      a.rot = (int)rope->rot_dim;
      kind = rope->interleaved ? 2 : 1;
    }
  }
  a.q_out = q_out;
  a.k_out = k_out;
  int fmt = 0;
  if (cache) {
    fmt = cache->fmt == FP8B_FMT_E5M2 ? 1 : 2;
    a.slots = slots;
    a.k_codes = cache->k_codes;
    a.v_codes = cache->v_codes;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.page_stride = cache->page_stride;
    a.scale_page_stride = cache->scale_page_stride;
    a.total_slots = cache->pages * cache->page_size;
    a.page_shift = __builtin_ctzll((unsigned long long)cache->page_size);
  }
  const int lpr = D <= 64 ? 8 : (D <= 128 ? 16 : 32);
  const int wg_slots = 256 / lpr;
  const int rows = q.heads + k.heads + v.heads;
  int shift = 0;
  while ((1 << shift) < rows && (1 << shift) < wg_slots) ++shift;
  a.slot_shift = shift;
  const int tokens = wg_slots >> shift;
  const int turns = (rows + (1 << shift) - 1) >> shift;
  int64_t gx = (T + tokens - 1) / tokens, gy = 1;
  a.items = turns;
  a.token_items = 1;
  if (gx < kManyWgs) {  // few tokens: every row a slot of its own
    gy = turns;
    a.items = 1;
  } else if (turns == 1 && kind == 0) {
    a.items = a.token_items = kTokenItems;
    gx = (T + (int64_t)tokens * kTokenItems - 1) / (tokens * kTokenItems);
  }
  const dim3 grid((unsigned)gx, (unsigned)gy);
#define FP8A_QKV(L, R, F) hipLaunchKernelGGL((qkv_kernel<L, R, F>), grid, dim3(256), 0, s, a)
#define FP8A_QKV_F(L, R)            \
  do {                              \
    if (fmt == 0) FP8A_QKV(L, R, 0); \
    else if (fmt == 1) FP8A_QKV(L, R, 1); \
    else FP8A_QKV(L, R, 2);         \
  } while (0)
#define FP8A_QKV_R(L)               \
  do {                              \
    if (kind == 0) FP8A_QKV_F(L, 0); \
    else if (kind == 1) FP8A_QKV_F(L, 1); \
    else FP8A_QKV_F(L, 2);          \
  } while (0)
  if (lpr == 8) FP8A_QKV_R(8);
  else if (lpr == 16) FP8A_QKV_R(16);
  else FP8A_QKV_R(32);
#undef FP8A_QKV_R
#undef FP8A_QKV_F
#undef FP8A_QKV
  return check_launch();
}

// ---- reading back ----------------------------------------------------------

struct ReadArgs {
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  int64_t page_stride, scale_page_stride, pages;
  int page_shift, heads, D;
  const int32_t* table;
  int64_t ld_table, cols;
  const int32_t* offsets;
  int64_t B, R;
  uint16_t *k_out, *v_out;
  uint32_t inv;    // ceil(2^32 / (D / 16)): divides a piece index by multiplication
  int slot_shift;  // log2 of the threads that share a row
};

constexpr int kReadRows = 16;  // rows per workgroup

// 16 rows per workgroup, K and V in blockIdx.y.  The first 16 threads look up
// each row's sequence (binary search over offsets) and page and leave them in
// LDS; then 2^slot_shift threads share a row, 16 codes each per turn (one
// 16-byte load, two 16-byte stores).  HBM-bound: 1 byte in, 2 out.
template <int FMT>
__global__ __launch_bounds__(256) void cache_read_kernel(const ReadArgs a) {
  __shared__ int64_t where_page[kReadRows];
  __shared__ int where_place[kReadRows];
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  const bool is_v = blockIdx.y != 0;
  if (tid < kReadRows) {
    const int64_t row = row0 + tid;
    int64_t page = -1;
    int place = 0;
    if (row < a.R && row < a.offsets[a.B]) {
      int64_t lo = 0, hi = a.B;  // offsets[lo] <= row < offsets[hi]
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= row) lo = mid;
        else hi = mid;
      }
      const int64_t tok = max(row - (int64_t)a.offsets[lo], (int64_t)0);
      const int64_t col = min(tok >> a.page_shift, a.cols - 1);
      page = a.table[lo * a.ld_table + col];
      page = page < 0 ? 0 : (page >= a.pages ? a.pages - 1 : page);
      place = (int)(tok & ((1 << a.page_shift) - 1));
    }
    where_page[tid] = page;
    where_place[tid] = place;
  }
  __syncthreads();
  const uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  const float* scales = is_v ? a.v_scales : a.k_scales;
  uint16_t* out = is_v ? a.v_out : a.k_out;
  const int per_head = a.D / 16;
  const int pieces = a.heads * per_head;
  const int share = 1 << a.slot_shift;
  const int groups = 256 >> a.slot_shift;
  for (int rr = tid >> a.slot_shift; rr < kReadRows; rr += groups) {
    const int64_t page = where_page[rr];
    if (page < 0) continue;
    const int place = where_place[rr];
    uint16_t* dst = out + (row0 + rr) * (int64_t)a.heads * a.D;
    for (int p = tid & (share - 1); p < pieces; p += share) {
      const int h = a.inv ? (int)__umulhi((uint32_t)p, a.inv) : p;
      const int c = p - h * per_head;
      const int64_t in_page = ((int64_t)h << a.page_shift) + place;
      const u32x4 raw =
          __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + page * a.page_stride + in_page * a.D + 16 * c));
      const float d = scales[page * a.scale_page_stride + in_page];
      u32x4 o[2];
      typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 lo, hi;
        if (FMT == 1) {
          lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8((int)raw[i], 1.0f, false);
          hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8((int)raw[i], 1.0f, true);
        } else {
          lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)raw[i], 1.0f, false);
          hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)raw[i], 1.0f, true);
        }
        const bf16x2 b0 = {(__bf16)(lo[0] * d), (__bf16)(lo[1] * d)};
        const bf16x2 b1 = {(__bf16)(hi[0] * d), (__bf16)(hi[1] * d)};
        o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, b0);
        o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, b1);
      }
      u32x4* d4 = reinterpret_cast<u32x4*>(dst + 16 * p);
      __builtin_nontemporal_store(o[0], d4);
      __builtin_nontemporal_store(o[1], d4 + 1);
    }
  }
}

int launch_cache_read(const fp8b_kv_cache& c, const int32_t* table, int64_t ld_table, int64_t cols,
                      const int32_t* offsets, int64_t B, int64_t R, uint16_t* k_out, uint16_t* v_out, hipStream_t s) {
  ReadArgs a{};
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.page_stride = c.page_stride;
  a.scale_page_stride = c.scale_page_stride;
  a.pages = c.pages;
  a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  a.heads = (int)c.heads;
  a.D = (int)c.head_dim;
  a.table = table;
  a.ld_table = ld_table;
  a.cols = cols;
  a.offsets = offsets;
  a.B = B;
  a.R = R;
  a.k_out = k_out;
  a.v_out = v_out;
  const uint32_t per_head = (uint32_t)a.D / 16;
  // p * inv >> 32 = p / per_head for p < 2^16: the excess of inv, below
  // per_head / 2^32 per unit, stays under 1 / per_head for those p
  a.inv = per_head == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + per_head - 1) / per_head);
  const int pieces = a.heads * (int)per_head;
  int shift = 0;
  while ((1 << shift) < pieces && shift < 8) ++shift;
  a.slot_shift = shift;
  const dim3 grid((unsigned)((R + kReadRows - 1) / kReadRows), 2);
  if (c.fmt == FP8B_FMT_E5M2) hipLaunchKernelGGL(cache_read_kernel<1>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(cache_read_kernel<2>, grid, dim3(256), 0, s, a);
  return check_launch();
}

}  // namespace fp8attn

// cache.hip -- what surrounds the attention kernel on a paged FP8 cache
// (layout: fp8b_kv_cache in include/fp8attn.h): query/key norms with the
// position rotation, the quantising write, and reading back.
#include "../csrc/common.hpp"
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
  float eps, inv_D;
  Rows q_out, k_out;
  const int64_t* slots;
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  uint32_t page_stride, scale_page_stride;
  int64_t total_slots;
  int page_shift;
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

// Global memory by its address (a plain pointer made of an integer would be
// accessed as if it might be LDS).
template <typename T>
using global_ptr = __attribute__((address_space(1))) T*;

__device__ __forceinline__ int64_t address(const void* p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }

// q, k or v by the row's number.
template <typename T>
__device__ __forceinline__ T of_kind(int row, int k0, int v0, T q, T k, T v) {
  return row < k0 ? q : (row < v0 ? k : v);
}

// Head h's 8 values of this lane; p: head 0's, step: bytes from head to head.
template <bool STREAM>
__device__ __forceinline__ u32x4 load_row(int64_t p, uint32_t step, int h, bool on) {
  const auto x = (global_ptr<const u32x4>)(p + (int64_t)((uint64_t)(uint32_t)h * step));
  u32x4 w = {0, 0, 0, 0};
  if (on) w = STREAM ? __builtin_nontemporal_load(x) : *x;
  return w;
}

// Codes and scale of a row of bf16 values (the quantiser of fp8_kv_quant and
// fp8_act_quant).  FMT 1: E5M2, 2: E4M3.
template <int LPR, int FMT>
__device__ __forceinline__ u32x2 quantise_row(const u32x4& raw, float& d) {
  constexpr float kMax = FMT == 1 ? 57344.0f : 448.0f;
  float f[8], v[8];
  unpack8(raw, f);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = row_max_nonneg<LPR>(amax);
  d = block_scale(amax, kMax, 1.0f / kMax);
  const BlockDivisor bd = make_divisor(amax, d);
  divide_block(f, v, bd);
  // With a normal d the quotients end at kMax (1 + 2^-23), which rounds to
  // kMax: only a subnormal d, rounded coarsely, needs the clamp.  By comparisons:
  // NaN passes, as it does on the other path (fminf and fmaxf would drop it).
  if (!bd.fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] > kMax ? kMax : (v[i] < -kMax ? -kMax : v[i]);
  }
  if (FMT == 1) return u32x2{pack4_e5m2(v[0], v[1], v[2], v[3]), pack4_e5m2(v[4], v[5], v[6], v[7])};
  return u32x2{pack4_e4m3(v[0], v[1], v[2], v[3]), pack4_e4m3(v[4], v[5], v[6], v[7])};
}

// One row (token, head) per LPR lanes, 8 values per lane, LPR * 8 >= D; the
// lanes past D hold zeros.  A workgroup's 256 / LPR row slots are split into
// groups of 2^slot_shift that share a token; rows are numbered queries, keys,
// values.  A slot takes `items` rows, the next one loaded while this one is
// worked on: other heads of its token, whose cos and sin it keeps, or
// (nothing to rotate, heads no more than slots) the same head of later tokens.
//
// FMT: 0 no cache (keys to k_out), 1 E5M2, 2 E4M3.  ROPE: 0 none, 1 halves,
// 2 interleaved.  STREAM: non-temporal loads.  HBM-bound (2 bytes in and 2, or
// 1 and a scale, out per value), but only just: 8 values are one 16-byte load
// and some 150 instructions, so addresses are kept to 32-bit products.  Norm
// and rotation of 4096 tokens x (64 + 8) x 128: 30.6 us, 5.0 TB/s; with the cache
// write of their keys and values 35.5 us (40.9 in two calls); cache write of 32768 x
// 8 x 128: 40 us, 5.1 TB/s; of one step's 32 tokens 2.3 us, which is the launch.
// (Times in this file: us a call in a replayed graph of calls on three sets of
// inputs in turn.)
template <int LPR, int ROPE, int FMT, bool STREAM>
__global__ __launch_bounds__(256) void qkv_kernel(const QkvArgs a) {
  constexpr int kSlots = 256 / LPR;
  const int lane = threadIdx.x & (LPR - 1);
  const int slot = threadIdx.x / LPR;
  const int per_token = 1 << a.slot_shift;
  const int tokens = kSlots >> a.slot_shift;  // of a workgroup at a time
  const int k0 = a.q.heads, v0 = a.q.heads + a.k.heads, rows = v0 + a.v.heads;
  int64_t t = (int64_t)blockIdx.x * tokens * a.token_items + (slot >> a.slot_shift);
  int r = (int)blockIdx.y * per_token + (slot & (per_token - 1));
  const int row_step = (int)gridDim.y * per_token;
  if (t >= a.T || r >= rows) return;
  const int e0 = 8 * lane;
  const bool on = e0 < a.D;
  const int half = a.rot >> 1;

  // Rows of this token, by kind.  Chosen by value: a choice of variables or of
  // the arguments' structs would be memory accesses.
  const int64_t qp = address(a.q.p) + 2 * (t * a.q.t + e0);
  int64_t kp = address(a.k.p) + 2 * (t * a.k.t + e0), vp = address(a.v.p) + 2 * (t * a.v.t + e0);
  const uint32_t qs = 2 * (uint32_t)a.q.h, ks = 2 * (uint32_t)a.k.h, vs = 2 * (uint32_t)a.v.h;
  const int64_t qo = address(a.q_out.p) + 2 * (t * a.q_out.t + e0);
  const int64_t ko = address(a.k_out.p) + 2 * (t * a.k_out.t + e0);
  u32x4 next = load_row<STREAM>(of_kind(r, k0, v0, qp, kp, vp), of_kind(r, k0, v0, qs, ks, vs),
                                 r - of_kind(r, k0, v0, 0, k0, v0), on);
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
      }
    } else if (e0 < a.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = tab[(e0 >> 1) + i];
        sn[i] = tab[half + (e0 >> 1) + i];
      }
    }
  }

  for (int left = a.items;; --left) {
    u32x4 raw = next;
    const int64_t sl = next_slot;
    const int rr = r;
    if (a.token_items > 1) {
      t += tokens;
      kp += 2 * tokens * a.k.t;  // (no queries and no k_out in a launch that walks along tokens)
      vp += 2 * tokens * a.v.t;
    } else {
      r += row_step;
    }
    const bool last = left == 1 || t >= a.T || r >= rows;
    if (!last) {
      next = load_row<STREAM>(of_kind(r, k0, v0, qp, kp, vp), of_kind(r, k0, v0, qs, ks, vs),
                               r - of_kind(r, k0, v0, 0, k0, v0), on);
      if (FMT != 0 && a.token_items > 1) next_slot = a.slots[t];
    }
    const int h = rr - of_kind(rr, k0, v0, 0, k0, v0);
    const uint16_t* w = rr < k0 ? a.q_weight : a.k_weight;
    if ((FMT == 0 || rr < v0) && (ROPE != 0 || w != nullptr)) {
      float f[8];
      unpack8(raw, f);
      if (w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
        ss = row_sum<LPR>(ss);
        // 1 / sqrt(mean + eps): the estimate (1 ulp) and one Newton step
        const float x = __builtin_fmaf(ss, a.inv_D, a.eps);
        const float y = __builtin_amdgcn_rsqf(x);
        const float rn = __builtin_fmaf(0.5f * y, __builtin_fmaf(-x * y, y, 1.0f), y);
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
        // positions past rot stay as they are, infinities too
        if (e0 < a.rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __builtin_fmaf(f[i], cs[i], o[i] * sn[i]);
        }
      } else if (ROPE == 2 && e0 < a.rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = f[2 * i], y = f[2 * i + 1];
          f[2 * i] = __builtin_fmaf(x, cs[i], -(y * sn[i]));
          f[2 * i + 1] = __builtin_fmaf(y, cs[i], x * sn[i]);
        }
      }
      raw = pack8(f);  // one rounding to bf16
    }
    if (FMT == 0 || rr < k0) {
      const uint32_t step = 2 * (uint32_t)(rr < k0 ? a.q_out.h : a.k_out.h);
      if (on) *(global_ptr<u32x4>)((rr < k0 ? qo : ko) + (int64_t)((uint64_t)(uint32_t)h * step)) = raw;
    } else if (sl >= 0 && sl < a.total_slots) {
      float d;
      const u32x2 codes = quantise_row<LPR, FMT>(raw, d);
      const uint32_t page = (uint32_t)(sl >> a.page_shift);
      const uint32_t in_page = ((uint32_t)h << a.page_shift) + ((uint32_t)sl & ((1u << a.page_shift) - 1));
      const int64_t cp = (rr < v0 ? address(a.k_codes) : address(a.v_codes)) +
                         (int64_t)((uint64_t)page * a.page_stride + in_page * (uint32_t)a.D);
      const int64_t sp = (rr < v0 ? address(a.k_scales) : address(a.v_scales)) +
                         4 * (int64_t)((uint64_t)page * a.scale_page_stride + in_page);
      if (on) *(global_ptr<u32x2>)(cp + e0) = codes;
      if (lane == 0) *(global_ptr<float>)sp = d;
    }
    if (last) return;
  }
}

// From 1024 workgroups of one token group each on, a slot takes several rows
// (rotation of 4096 x 72 heads: 31 us, 40 with a slot for every row; write of 900
// tokens x 8 heads: 3.2 us, 4.5 with several rows a slot).  512: rotation of 512 x 72
// 7.0 -> 8.0 us; 2048: 1500 x 72 12.1 -> 13.9.
constexpr int kManyWgs = 1024;
// Rows that the last-level cache (256 MB) can still hold are read from there: a
// write of 134 MB of rows (32768 x 8 heads) 45.4 us with plain loads, 42.0
// non-temporal; of 17 MB 7.5 and 7.9.
constexpr int64_t kStreamBytes = (int64_t)64 << 20;
// Tokens a slot takes in a large cache write: 32768 x 8 heads 44.6 us with 1, 39.7
// with 2, 39.4 with 4, 39.9 with 8; 4096 x 8 7.2, -, 7.3, 8.9.
constexpr int kTokenItems = 4;

int launch_qkv(const Rows& q, const Rows& k, const Rows& v, int64_t T, int D, const fp8b_rope* rope, const Rows& q_out,
               const Rows& k_out, const int64_t* slots, const fp8b_kv_cache* cache, hipStream_t s) {
  QkvArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.T = T;
  a.D = D;
  a.inv_D = 1.0f / (float)D;
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
    a.page_stride = (uint32_t)cache->page_stride;
    a.scale_page_stride = (uint32_t)cache->scale_page_stride;
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
  } else if (turns == 1 && kind == 0 && q.heads == 0) {
    a.items = a.token_items = kTokenItems;
    gx = (T + (int64_t)tokens * kTokenItems - 1) / (tokens * kTokenItems);
  }
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const bool streamed = kind == 0 && cache && 2 * T * rows * D >= kStreamBytes;
#define FP8A_QKV(L, R, F) hipLaunchKernelGGL((qkv_kernel<L, R, F, false>), grid, dim3(256), 0, s, a)
#define FP8A_QKV_S(L, F) hipLaunchKernelGGL((qkv_kernel<L, 0, F, true>), grid, dim3(256), 0, s, a)
#define FP8A_QKV_F(L, R)                      \
  do {                                        \
    if (fmt == 0) FP8A_QKV(L, R, 0);          \
    else if (R == 0 && streamed && fmt == 1) FP8A_QKV_S(L, 1); \
    else if (R == 0 && streamed) FP8A_QKV_S(L, 2); \
    else if (fmt == 1) FP8A_QKV(L, R, 1);     \
    else FP8A_QKV(L, R, 2);                   \
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
#undef FP8A_QKV_S
#undef FP8A_QKV
  return check_launch();
}

// ---- reading back ----------------------------------------------------------

// x / d for x < 2^16 and inv = ceil(2^32 / d) (d = 1: inv 0): the excess of inv,
// below d / 2^32 per unit, adds up to less than 1 / d.
__device__ __forceinline__ int divide_by(int x, uint32_t inv) { return inv ? (int)__umulhi((uint32_t)x, inv) : x; }
static uint32_t inverse(uint32_t d) { return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }

struct ReadArgs {
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  uint32_t page_stride, scale_page_stride;
  int64_t pages;
  int page_shift, heads, D;
  const int32_t* table;
  int64_t ld_table, cols;
  const int32_t* offsets;
  int64_t B, R;
  uint16_t *k_out, *v_out;
  int rows;                       // of a workgroup
  uint32_t inv_pieces, inv_head;  // of the pieces of a row and of a head
};

constexpr int kReadTurns = 2;       // pieces a thread takes, all loaded before any is put out
constexpr int kReadPieces = 256 * kReadTurns;

// A workgroup takes `rows` rows, their pieces of 16 codes (one 16-byte load,
// two 16-byte stores) dealt to the threads in one line: as many rows as fill
// 512 pieces, or one longer row in turns; K and V in blockIdx.y.  Its threads
// first look up each row's sequence (binary search over offsets) and page and
// leave them in LDS.  HBM-bound: 1 byte in, 2 out: 32768 tokens x 8 x 128, K and
// V, 41.2 us, 4.9 TB/s (one piece a turn 42.9, four 43.7, eight 44.8).  Rows and
// pieces that do not exist are read at valid addresses and not put out, so that
// no branch comes between the loads.
template <int FMT>
__global__ __launch_bounds__(256) void cache_read_kernel(const ReadArgs a) {
  __shared__ int row_page[kReadPieces];  // -1: no such row
  __shared__ int row_place[kReadPieces];
  const int tid = threadIdx.x;
  const int rows = a.rows;
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const bool is_v = blockIdx.y != 0;
  for (int x = tid; x < rows; x += 256) {
    const int64_t row = row0 + x;
    int page = -1, place = 0;
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
      page = page < 0 ? 0 : (page >= a.pages ? (int)a.pages - 1 : page);
      place = (int)(tok & ((1 << a.page_shift) - 1));
    }
    row_page[x] = page;
    row_place[x] = place;
  }
  __syncthreads();
  const uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  const float* scales = is_v ? a.v_scales : a.k_scales;
  uint16_t* out = (is_v ? a.v_out : a.k_out) + row0 * a.heads * a.D;
  const int per_head = a.D / 16;
  const int pieces = a.heads * per_head, total = rows * pieces;
  for (int i0 = tid; i0 < ((total + kReadPieces - 1) & ~(kReadPieces - 1)); i0 += kReadPieces) {
    u32x4 raw[kReadTurns];
    float d[kReadTurns];
    int to[kReadTurns];  // piece of the output, -1: none
#pragma unroll
    for (int u = 0; u < kReadTurns; ++u) {
      const int i = min(i0 + 256 * u, total - 1);
      const int x = rows == 1 ? 0 : divide_by(i, a.inv_pieces);
      const int p = i - x * pieces;
      const int h = divide_by(p, a.inv_head);
      to[u] = row_page[x] >= 0 && i0 + 256 * u < total ? i : -1;
      const uint32_t page = (uint32_t)max(row_page[x], 0);
      const uint32_t in_page = ((uint32_t)h << a.page_shift) + (uint32_t)row_place[x];
      raw[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
          codes + ((uint64_t)page * a.page_stride + in_page * (uint32_t)a.D + 16 * (p - h * per_head))));
      d[u] = scales[(uint64_t)page * a.scale_page_stride + in_page];
    }
#pragma unroll
    for (int u = 0; u < kReadTurns; ++u) {
      u32x4 o[2];
      typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 lo, hi;
        if (FMT == 1) {
          lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8((int)raw[u][i], 1.0f, false);
          hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8((int)raw[u][i], 1.0f, true);
        } else {
          lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)raw[u][i], 1.0f, false);
          hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)raw[u][i], 1.0f, true);
        }
        const bf16x2 b0 = {(__bf16)(lo[0] * d[u]), (__bf16)(lo[1] * d[u])};
        const bf16x2 b1 = {(__bf16)(hi[0] * d[u]), (__bf16)(hi[1] * d[u])};
        o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, b0);
        o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, b1);
      }
      if (to[u] >= 0) {
        u32x4* q = reinterpret_cast<u32x4*>(out + (int64_t)16 * to[u]);
        __builtin_nontemporal_store(o[0], q);
        __builtin_nontemporal_store(o[1], q + 1);
      }
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
  a.page_stride = (uint32_t)c.page_stride;
  a.scale_page_stride = (uint32_t)c.scale_page_stride;
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
  const int pieces = a.heads * (a.D / 16);
  a.rows = pieces < kReadPieces ? kReadPieces / pieces : 1;
  a.inv_pieces = inverse((uint32_t)pieces);
  a.inv_head = inverse((uint32_t)a.D / 16);
  const dim3 grid((unsigned)((R + a.rows - 1) / a.rows), 2);
  if (c.fmt == FP8B_FMT_E5M2) hipLaunchKernelGGL(cache_read_kernel<1>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(cache_read_kernel<2>, grid, dim3(256), 0, s, a);
  return check_launch();
}

}  // namespace fp8attn

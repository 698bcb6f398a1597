// paged.hip -- attention of one new token per sequence over a paged FP8
// key-value cache (include/fp8attn.h, fp8_paged_attention).
//
// The work is reading the cache: per token and KV head 2 D bytes of codes
// and two scales, for 4 D G operations (G query heads share a KV head), so
// HBM bounds it as long as the arithmetic keeps up.  One wave takes 32 tokens
// at a time straight from memory into registers, with no LDS on the way:
//
//   S^T = K Q^T   v_mfma_f32_16x16x32_bf16, keys as rows, query heads as
//                 columns (G <= 16 of them; more take further tiles).  Lane
//                 (g, r) = (lane / 16, lane % 16) loads 16-byte pieces g of
//                 key r; which of the D positions a product's k index means
//                 is free as long as K and Q agree, so the pieces are taken
//                 as they lie.
//   softmax       lane (g, c) then holds head c's scores of keys 4g .. 4g+3
//                 of each 16: running maximum per head (two lane swaps),
//                 accumulators rescaled only when a maximum grows, sums kept
//                 per lane and joined at the end.
//   O^T = V^T P^T the same lane's 8 weights are the product's B operand as
//                 they lie.  Lane (g, r) loads D/16 adjacent bytes of those 8
//                 keys' V rows, so its A operand is an 8 x D/16 byte
//                 transpose in registers: v_perm pairs two keys' bytes,
//                 v_cvt_scalef32_pk_bf16 widens the pair.
//
// Codes are exact in bf16 and Q is bf16, so S is exact but for fp32 sums.
// The weights (times the V scale) are split into 2 bf16 terms for bf16
// output and 3 for fp32 output: one term alone would be as coarse as the
// output's own rounding; the further MFMAs are hidden behind the loads.
#include "../common.hpp"
#include "attn_launch.hpp"

namespace fp8attn {

using namespace fp8blk;

constexpr int kTile = 32;       // keys a wave takes at a time
constexpr int kWaves = 4;       // waves of a workgroup
constexpr int kMaxWgs = 1024;   // workgroups of a split launch: 4 for each of the 256 CUs
constexpr int kMinTiles = 8;    // tiles (all waves together) a workgroup of a split launch takes at least

struct AttnArgs {
  const uint16_t* q;
  int64_t q_b, q_h;
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  int64_t k_page_stride, v_page_stride, k_scale_page_stride, v_scale_page_stride;
  int pages, page_shift, heads, D;
  int G, qtiles;  // query heads per KV head, and how many 16-row tiles they take
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int B, Hq, max_len, window;
  float scale_log2e;
  void* out;
  int out_f32;
  float* lse;
  float* ws;
  int split;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The tokens a sequence's new token sees, [lo, n), and the tiles (aligned to
// 32) they lie in.  A sequence that sees nothing counts one tile, which reads
// nothing and puts out the empty row.
struct Span {
  int lo, n, tile0, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  Span s;
  const int len = a.lens[b];
  s.n = len < 0 ? 0 : (len < a.max_len ? len : a.max_len);
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.tile0 = s.lo / kTile;
  const int end = (s.n + kTile - 1) / kTile;
  s.tiles = end > s.tile0 ? end - s.tile0 : 1;
  return s;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The work of a launch is the line of all tiles: sequences in order, each
// one's regions (KV head, query tile) in order, each region's tiles in order.
// Total tiles, or (find) the sequence that holds tile t and where it begins.
__device__ __forceinline__ int total_tiles(const AttnArgs& a) {
  const int lane = threadIdx.x & 63, R = a.heads * a.qtiles;
  int sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    sum += b < a.B ? span_of(a, b).tiles * R : 0;
  }
  return uniform(wave_sum(sum));
}
__device__ __forceinline__ void find_tile(const AttnArgs& a, int t, int& seq, int& begin) {
  const int lane = threadIdx.x & 63, R = a.heads * a.qtiles;
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    const int v = b < a.B ? span_of(a, b).tiles * R : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      incl += lane >= o ? u : 0;
    }
    const int all = __builtin_amdgcn_readlane(incl, 63);
    if (t < base + all) {
      const unsigned long long past = __ballot(base + incl <= t);  // sequences that end at or before t
      const int k = __popcll(past);
      seq = uniform(b0 + k);
      begin = base + __builtin_amdgcn_readlane(incl - v, uniform(k));
      return;
    }
    base += all;
  }
  seq = a.B;
  begin = base;
}
// Where sequence b begins on the line.
__device__ __forceinline__ int begin_of(const AttnArgs& a, int b) {
  const int lane = threadIdx.x & 63, R = a.heads * a.qtiles;
  int sum = 0;
  for (int b0 = 0; b0 < b; b0 += 64) sum += b0 + lane < b ? span_of(a, b0 + lane).tiles * R : 0;
  return uniform(wave_sum(sum));
}
__device__ __forceinline__ int tiles_per_wg(int total, int wgs) {
  const int per = (total + wgs - 1) / wgs;
  return per > kMinTiles ? per : kMinTiles;
}

// Floats of a partial result: G rows of D, then G maxima, then G sums.
__host__ __device__ inline int64_t partial_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// Two codes (the low or high half of w) as exact bf16.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if (FMT == 1) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)w, 1.0f, HI));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI));
}

__device__ __forceinline__ float swap_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// Where a region's rows of a half tile (16 keys, all in one page) lie.
struct Bases {
  const uint8_t *k, *v;
  const float *ks, *vs;
};
struct Half {
  int page, place;  // place: of the first key, a multiple of 16
};

// What a wave holds of a tile of 32 keys, per half u of 16: K pieces (16
// bytes of each 64 positions) of key r, V words of keys 4g .. 4g+3, and
// those keys' scales.
template <int DP>
struct KeyRegs {
  u32x4 c[2][DP / 64];
  v4f s[2];
};
template <int DP>
struct ValueRegs {
  uint32_t c[2][4][DP / 64];
  v4f s[2];
};

template <int DP, bool FULL>
__device__ __forceinline__ void load_keys(const AttnArgs& a, const Bases& at, const Half (&hf)[2], KeyRegs<DP>& k) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int D = FULL ? DP : a.D;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* p = at.k + (hf[u].page * a.k_page_stride + hf[u].place * D);
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      // pieces past D are read from the row's start and zeroed before use
      const int off = FULL || 64 * c + 16 * g < D ? 64 * c + 16 * g : 0;
      k.c[u][c] = *reinterpret_cast<const u32x4*>(p + (uint32_t)(r * D + off));
    }
    const float* q = at.ks + (hf[u].page * a.k_scale_page_stride + hf[u].place);
    k.s[u] = *reinterpret_cast<const v4f*>(q + 4 * g);
  }
}

template <int DP, bool FULL>
__device__ __forceinline__ void load_values(const AttnArgs& a, const Bases& at, const Half (&hf)[2],
                                            ValueRegs<DP>& v) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int D = FULL ? DP : a.D;
  constexpr int W = DP / 64;
  const int d0 = FULL || 4 * W * r < D ? 4 * W * r : 0;  // lanes past D: their positions are not put out
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* p = at.v + (hf[u].page * a.v_page_stride + hf[u].place * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t* x = reinterpret_cast<const uint32_t*>(p + (uint32_t)((4 * g + i) * D + d0));
      if (W == 4) {
        const u32x4 y = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
        for (int w = 0; w < W; ++w) v.c[u][i][w] = y[w];
      } else if (W == 2) {
        const u32x2 y = *reinterpret_cast<const u32x2*>(x);
#pragma unroll
        for (int w = 0; w < W; ++w) v.c[u][i][w] = y[w];
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) v.c[u][i][w] = x[w];
      }
    }
    const float* q = at.vs + (hf[u].page * a.v_scale_page_stride + hf[u].place);
    v.s[u] = *reinterpret_cast<const v4f*>(q + 4 * g);
  }
}

// Running state of a wave: per lane (g, c) the maximum of head c (log2
// domain), this lane's part of its sum, and O^T: o[j][i] is head c, position
// (DP/16)(4g + i) + j.
template <int DP>
struct State {
  float m, l;
  v4f o[DP / 16];
};

// s = K Q^T with scales, log2 domain.
template <int DP, bool FULL, int FMT>
__device__ __forceinline__ void scores(const AttnArgs& a, const bf16x8 (&qf)[DP / 32], const KeyRegs<DP>& k,
                                       float (&s)[8]) {
  const int g = (threadIdx.x & 63) >> 4;
  typedef uint32_t frag __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      u32x4 w = k.c[u][c];
      if (!FULL && 64 * c + 16 * g >= a.D) w = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const frag kf = {widen2<FMT, false>(w[2 * x]), widen2<FMT, true>(w[2 * x]), widen2<FMT, false>(w[2 * x + 1]),
                         widen2<FMT, true>(w[2 * x + 1])};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf), qf[2 * c + x], acc, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[4 * u + i] = acc[i] * (k.s[u][i] * a.scale_log2e);
  }
}

// The weights of a tile's scores, the running maximum and sum brought up to
// date.
template <int DP>
__device__ __forceinline__ void weights(float (&s)[8], State<DP>& st) {
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
  mx = swap_max(mx);
  if (__any(mx > st.m)) {
    const float m = fmaxf(st.m, mx);
    // m is -inf only where nothing was seen yet: nothing to rescale
    const float alpha = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= alpha;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[j][i] *= alpha;
  }
  const float m = st.m == -__builtin_inff() ? 0.0f : st.m;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = __builtin_amdgcn_exp2f(s[i] - m);
    st.l += s[i];
  }
}

// O += P V, p the weights times the V scales.
template <int DP, int FMT, int TERMS>
__device__ __forceinline__ void accumulate(float (&p)[8], const ValueRegs<DP>& v, State<DP>& st) {
  typedef uint32_t frag __attribute__((ext_vector_type(4)));
  // p = sum of TERMS bf16 terms, each the rounded rest of those before
  bf16x8 pf[TERMS];
#pragma unroll
  for (int t = 0; t < TERMS; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pf[t][i] = (__bf16)p[i];
      p[i] -= (float)pf[t][i];
    }
#pragma unroll
  for (int w = 0; w < DP / 64; ++w) {
    // keys (0, 1) and (2, 3) of each half paired byte by byte
    uint32_t pr[2][2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t k0 = v.c[u][2 * y][w], k1 = v.c[u][2 * y + 1][w];
        pr[u][y][0] = __builtin_amdgcn_perm(k1, k0, 0x05010400u);
        pr[u][y][1] = __builtin_amdgcn_perm(k1, k0, 0x07030602u);
      }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      frag vf;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          vf[2 * u + y] = (b & 1) ? widen2<FMT, true>(pr[u][y][b >> 1]) : widen2<FMT, false>(pr[u][y][b >> 1]);
      const int j = 4 * w + b;
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        st.o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vf), pf[t], st.o[j], 0, 0, 0);
    }
  }
}

// A wave's tiles t, t + kWaves, ... below `end` (relative to the span's
// first) of one region.  The next tile's keys are loaded as soon as this
// one's are used, its values likewise: a tile is always in flight and needs
// no second set of registers.  The page of each half tile is looked up 32
// tiles ahead, one per lane.
template <int DP, bool FULL, int FMT, int TERMS>
__device__ __forceinline__ void run_tiles(const AttnArgs& a, const Span& sp, int b, int h,
                                          const bf16x8 (&qf)[DP / 32], int t, int end, State<DP>& st) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int32_t* row = a.table + b * a.ld_table;
  const int64_t head_row = (int64_t)h << a.page_shift;
  const Bases at = {a.k_codes + head_row * a.D, a.v_codes + head_row * a.D, a.k_scales + head_row,
                    a.v_scales + head_row};
  const int last = (sp.n - 1) >> 4;  // the last 16 tokens that hold one
  int ids = 0, ahead = t - 32 * kWaves;  // ids: pages of the 32 tiles from `ahead` on

  Half hf[2];
  auto locate = [&](int tt) {
    if (tt - ahead >= 32 * kWaves) {
      ahead = tt;
      const int grp = min(2 * (sp.tile0 + tt + (lane >> 1) * kWaves) + (lane & 1), last);
      ids = row[(grp << 4) >> a.page_shift];
      ids = ids < 0 ? 0 : (ids >= a.pages ? a.pages - 1 : ids);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      hf[u].page = __builtin_amdgcn_readlane(ids, 2 * ((tt - ahead) / kWaves) + u);
      hf[u].place = (min(2 * (sp.tile0 + tt) + u, last) << 4) & ((1 << a.page_shift) - 1);
    }
  };

  if (t >= end) return;
  KeyRegs<DP> k;
  ValueRegs<DP> v;
  locate(t);
  load_keys<DP, FULL>(a, at, hf, k);
  load_values<DP, FULL>(a, at, hf, v);
  for (;;) {
    const int next = t + kWaves;
    float s[8];
    scores<DP, FULL, FMT>(a, qf, k, s);
    if (next < end) {
      locate(next);
      load_keys<DP, FULL>(a, at, hf, k);
    }
    const int first = (sp.tile0 + t) * kTile;
    if (first < sp.lo || first + kTile > sp.n) {
      // nothing of a token that is not seen may reach a product
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = first + 16 * u + 4 * g + i;
          if (j < sp.lo || j >= sp.n) {
            s[4 * u + i] = -__builtin_inff();
            v.s[u][i] = 0.0f;
#pragma unroll
            for (int w = 0; w < DP / 64; ++w) v.c[u][i][w] = 0u;
          }
        }
    }
    weights<DP>(s, st);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= v.s[i >> 2][i & 3];
    accumulate<DP, FMT, TERMS>(s, v, st);
    if (next >= end) return;
    load_values<DP, FULL>(a, at, hf, v);
    t = next;
  }
}

// One workgroup takes a piece of the line (split) or one region (not split).
// In a piece, each region's tiles are dealt to the four waves, whose results
// are joined in LDS; a region that lies whole in the piece is put out, others
// go to the workspace: slot 2w for the region the piece begins in, slot 2w+1
// for the one it ends in.
template <int DP, bool FULL, int FMT, int TERMS>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attend_kernel(const AttnArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int R = a.heads * a.qtiles;
  const int rows_max = a.G < 16 ? a.G : 16;
  constexpr int LD = DP + 4;
  float* lds_m = lds + (int64_t)kWaves * rows_max * LD;  // [wave][16]
  float* lds_l = lds_m + kWaves * 16;

  int b, region, tile, left;  // left: tiles of this piece still to do
  int piece0 = 0;             // where the piece begins on the line
  int seq_begin = 0;
  if (a.split) {
    const int total = total_tiles(a);
    const int per = tiles_per_wg(total, gridDim.x);
    piece0 = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
    left = min(per, total - piece0);
    if (left <= 0) return;
    find_tile(a, piece0, b, seq_begin);
  } else {
    b = blockIdx.x / R;
    region = blockIdx.x % R;
    tile = 0;
    left = 0x7fffffff;
  }
  Span sp = span_of(a, b);
  if (a.split) {
    region = (piece0 - seq_begin) / sp.tiles;
    tile = (piece0 - seq_begin) % sp.tiles;
  }

  for (;;) {
    const int count = min(sp.tiles - tile, left);
    const int h = uniform(region / a.qtiles), qt = uniform(region % a.qtiles);
    const int rows = min(16, a.G - 16 * qt);
    const int head0 = h * a.G + 16 * qt;
    State<DP> st;
    st.m = -__builtin_inff();
    st.l = 0.0f;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) st.o[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (sp.n > 0) {
      bf16x8 qf[DP / 32];
      const uint16_t* qp = a.q + b * a.q_b + (int64_t)(head0 + c) * a.q_h;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j) {
        const int d = 64 * (j >> 1) + 16 * g + 8 * (j & 1);
        u32x4 w = {0, 0, 0, 0};
        if (c < rows && (FULL || d < a.D)) w = *reinterpret_cast<const u32x4*>(qp + d);
        qf[j] = __builtin_bit_cast(bf16x8, w);
      }
      run_tiles<DP, FULL, FMT, TERMS>(a, sp, b, h, qf, tile + wave, tile + count, st);
    }
    st.l += __shfl_xor(st.l, 16);
    st.l += __shfl_xor(st.l, 32);
    if (c < rows) {
      float* o = lds + ((int64_t)wave * rows_max + c) * LD;
#pragma unroll
      for (int j = 0; j < DP / 16; j += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<v4f*>(o + (DP / 16) * (4 * g + i) + j) =
              v4f{st.o[j][i], st.o[j + 1][i], st.o[j + 2][i], st.o[j + 3][i]};
    }
    if (g == 0) {
      lds_m[wave * 16 + c] = st.m;
      lds_l[wave * 16 + c] = st.l;
    }
    __syncthreads();
    const bool whole = count == sp.tiles;
    float* part = nullptr;
    if (!whole) part = a.ws + (2 * (int64_t)blockIdx.x + (tile == 0 ? 1 : 0)) * partial_floats(rows_max, a.D);
    const int q4 = a.D / 4;
    for (int x = tid; x < rows * q4; x += 256) {
      const int rr = x / q4, d = 4 * (x - rr * q4);
      float m = lds_m[rr];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) m = fmaxf(m, lds_m[w * 16 + rr]);
      const float ms = m == -__builtin_inff() ? 0.0f : m;
      float l = 0.0f;
      v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(lds_m[w * 16 + rr] - ms);
        l = __builtin_fmaf(f, lds_l[w * 16 + rr], l);
        const v4f ow = *reinterpret_cast<const v4f*>(lds + ((int64_t)w * rows_max + rr) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(f, ow[i], o[i]);
      }
      if (whole) {
        const int64_t at = (int64_t)b * a.Hq + head0 + rr;
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= inv;
        if (a.out_f32) {
          *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at * a.D + d) = o;
        } else {
          const bf16x2 b0 = {(__bf16)o[0], (__bf16)o[1]}, b1 = {(__bf16)o[2], (__bf16)o[3]};
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * a.D + d) =
              u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
        }
        if (a.lse && d == 0) a.lse[at] = l > 0.0f ? (m + __log2f(l)) * 0.69314718056f : -__builtin_inff();
      } else {
        *reinterpret_cast<v4f*>(part + (int64_t)rr * a.D + d) = o;
        if (d == 0) {
          part[(int64_t)rows_max * a.D + rr] = m;
          part[(int64_t)rows_max * a.D + rows_max + rr] = l;
        }
      }
    }
    left -= count;
    tile = 0;
    if (!a.split || left <= 0) return;
    __syncthreads();  // the next region's results go to the same LDS
    if (++region == R) {
      region = 0;
      ++b;
      sp = span_of(a, b);
    }
  }
}

// Joins the partial results of each region that several pieces share: one
// workgroup per query head of a region (blockIdx.y the row).  Its threads are
// D/4 columns by as many groups of pieces as fit.
__global__ __launch_bounds__(256) void join_kernel(const AttnArgs a, int wgs) {
  __shared__ float lds[256 * 4 + 256];
  const int tid = threadIdx.x;
  const int R = a.heads * a.qtiles;
  const int b = blockIdx.x / R, region = blockIdx.x % R;
  const int h = region / a.qtiles, qt = region % a.qtiles;
  const int rr = blockIdx.y;
  if (rr >= min(16, a.G - 16 * qt)) return;
  const int rows_max = a.G < 16 ? a.G : 16;
  const int per = tiles_per_wg(total_tiles(a), wgs);
  const Span sp = span_of(a, b);
  const int t0 = begin_of(a, b) + region * sp.tiles, t1 = t0 + sp.tiles;
  const int w0 = t0 / per, w1 = (t1 - 1) / per;
  if (w0 == w1) return;  // put out by the piece that held it whole

  const int64_t pf = partial_floats(rows_max, a.D);
  const int q4 = a.D / 4, groups = 256 / q4;
  const int grp = tid / q4, d = 4 * (tid - grp * q4);
  float m = -__builtin_inff(), l = 0.0f;
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (grp < groups) {
    for (int w = w0 + grp; w <= w1; w += groups) {
      // the first of them ends its piece in the region, the others begin theirs
      const float* p = a.ws + (2 * (int64_t)w + (w == w0 ? 1 : 0)) * pf;
      const float pm = p[(int64_t)rows_max * a.D + rr], pl = p[(int64_t)rows_max * a.D + rows_max + rr];
      const v4f po = *reinterpret_cast<const v4f*>(p + (int64_t)rr * a.D + d);
      const float nm = fmaxf(m, pm), ns = nm == -__builtin_inff() ? 0.0f : nm;
      const float f0 = __builtin_amdgcn_exp2f(m - ns), f1 = __builtin_amdgcn_exp2f(pm - ns);
      m = nm;
      l = l * f0 + pl * f1;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f0 + po[i] * f1;
    }
    *reinterpret_cast<v4f*>(lds + 4 * tid) = o;
    if (d == 0) {
      lds[1024 + grp] = m;
      lds[1024 + 128 + grp] = l;
    }
  }
  __syncthreads();
  if (grp != 0) return;
  float mt = -__builtin_inff();
  for (int k = 0; k < groups; ++k) mt = fmaxf(mt, lds[1024 + k]);
  const float ms = mt == -__builtin_inff() ? 0.0f : mt;
  l = 0.0f;
  o = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < groups; ++k) {
    const float f = __builtin_amdgcn_exp2f(lds[1024 + k] - ms);
    l += f * lds[1024 + 128 + k];
    const v4f ok = *reinterpret_cast<const v4f*>(lds + 4 * (k * q4 + tid));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += f * ok[i];
  }
  const int64_t at = (int64_t)b * a.Hq + h * a.G + 16 * qt + rr;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  if (a.out_f32) {
    *reinterpret_cast<v4f*>(static_cast<float*>(a.out) + at * a.D + d) = o;
  } else {
    const bf16x2 b0 = {(__bf16)o[0], (__bf16)o[1]}, b1 = {(__bf16)o[2], (__bf16)o[3]};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * a.D + d) =
        u32x2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
  }
  if (a.lse && d == 0) a.lse[at] = l > 0.0f ? (mt + __log2f(l)) * 0.69314718056f : -__builtin_inff();
}

// ---- host -------------------------------------------------------------------

struct Shape {
  int G, qtiles, rows;
  int64_t regions, max_len, wgs;  // wgs: workgroups of a split launch; 0: one workgroup per region
};

static Shape shape_of(const fp8b_kv_cache& c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                      int64_t window) {
  Shape s;
  s.G = (int)(Hq / c.heads);
  s.qtiles = (s.G + 15) / 16;
  s.rows = s.G < 16 ? s.G : 16;
  s.regions = B * c.heads * s.qtiles;
  const int64_t room = cols * c.page_size;
  s.max_len = max_context < room ? max_context : room;
  // the most tiles a region can have: a window reaches into one more
  const int64_t seen = window > 0 && window < s.max_len ? window + kTile - 1 : s.max_len;
  const int64_t tiles = (seen + kTile - 1) / kTile;
  if (tiles <= kMinTiles) {
    s.wgs = 0;
  } else {
    const int64_t want = (s.regions * tiles + kMinTiles - 1) / kMinTiles;
    s.wgs = want < kMaxWgs ? want : kMaxWgs;
  }
  return s;
}

int64_t attention_workspace(const fp8b_kv_cache& c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                            int64_t window) {
  const Shape s = shape_of(c, B, Hq, cols, max_context, window);
  return 2 * s.wgs * partial_floats(s.rows, (int)c.head_dim) * (int64_t)sizeof(float);
}

template <int DP, bool FULL, int FMT, int TERMS>
static int launch_one(const AttnArgs& a, unsigned grid, hipStream_t s) {
  const int rows = a.G < 16 ? a.G : 16;
  const size_t lds = (size_t)(kWaves * rows * (DP + 4) + 2 * kWaves * 16) * sizeof(float);
  hipLaunchKernelGGL((attend_kernel<DP, FULL, FMT, TERMS>), dim3(grid), dim3(256), lds, s, a);
  return check_launch();
}
template <int DP, bool FULL>
static int launch_dp(const AttnArgs& a, int fmt, unsigned grid, hipStream_t s) {
  if (fmt == FP8B_FMT_E5M2)
    return a.out_f32 ? launch_one<DP, FULL, 1, 3>(a, grid, s) : launch_one<DP, FULL, 1, 2>(a, grid, s);
  return a.out_f32 ? launch_one<DP, FULL, 2, 3>(a, grid, s) : launch_one<DP, FULL, 2, 2>(a, grid, s);
}

int launch_attention(const fp8b_kv_cache& c, const Attention& p, hipStream_t s) {
  const Shape sh = shape_of(c, p.B, p.Hq, p.cols, p.max_context, p.window);
  AttnArgs a{};
  a.q = p.q;
  a.q_b = p.q_b;
  a.q_h = p.q_h;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.k_page_stride = c.k_page_stride;
  a.v_page_stride = c.v_page_stride;
  a.k_scale_page_stride = c.k_scale_page_stride;
  a.v_scale_page_stride = c.v_scale_page_stride;
  a.pages = (int)c.pages;
  a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  a.heads = (int)c.heads;
  a.D = (int)c.head_dim;
  a.G = sh.G;
  a.qtiles = sh.qtiles;
  a.table = p.table;
  a.ld_table = p.ld_table;
  a.lens = p.lens;
  a.B = (int)p.B;
  a.Hq = (int)p.Hq;
  a.max_len = (int)sh.max_len;
  a.window = (int)(p.window < sh.max_len ? p.window : 0);  // a window of max_len or more hides nothing
  a.scale_log2e = p.scale * 1.44269504089f;
  a.out = p.out;
  a.out_f32 = p.out_f32;
  a.lse = p.lse;
  a.ws = p.workspace;
  a.split = sh.wgs > 0;
  const unsigned grid = (unsigned)(sh.wgs > 0 ? sh.wgs : sh.regions);
  int rc;
  if (a.D == 64) rc = launch_dp<64, true>(a, c.fmt, grid, s);
  else if (a.D < 64) rc = launch_dp<64, false>(a, c.fmt, grid, s);
  else if (a.D == 128) rc = launch_dp<128, true>(a, c.fmt, grid, s);
  else if (a.D < 128) rc = launch_dp<128, false>(a, c.fmt, grid, s);
  else if (a.D == 192) rc = launch_dp<192, true>(a, c.fmt, grid, s);
  else if (a.D == 256) rc = launch_dp<256, true>(a, c.fmt, grid, s);
  else rc = launch_dp<256, false>(a, c.fmt, grid, s);
  if (rc != FP8B_OK || !a.split) return rc;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)sh.regions, (unsigned)sh.rows), dim3(256), 0, s, a, (int)grid);
  return check_launch();
}

}  // namespace fp8attn

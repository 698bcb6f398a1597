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
// The weights (times the V scale) are split into 3 bf16 terms, which hold all
// 24 bits of them: nothing before the output's own rounding is coarser than
// fp32 (2 terms, 16 bits, gave bf16 outputs that are off by a rounding where V
// lies within 2^-16 of a tie).
//
// Times in this file: us a call on the GPU in a replayed graph of calls on three
// sets of inputs in turn, E5M2 and bf16 output if nothing else is said; a copy of
// 200 MB runs at 5.4 TB/s.
//
// Measured (128 positions, lengths from half to one and a half times the average):
// 128 sequences x 6000 tokens x 8 heads for 64 query heads 306 us (5.2 TB/s), one of
// 131072 tokens x 8 heads 60 (4.6 TB/s), 32 x 2048 x 8 33 (27, 4.6 TB/s, when all are
// equally long: a workgroup a region waits for the longest), 8 x 1000 x 8 11.3, 129
// tokens x 8 5.4.  A tile takes 281 vector instructions and 32 MFMAs, about 0.75 us of
// a SIMD that has one wave: at the memory's rate two fifths of the vector units'
// time.  Short contexts are bound by each workgroup's chain of loads.
#include <type_traits>

#include "../csrc/common.hpp"
#include "attn_launch.hpp"

namespace fp8attn {

using namespace fp8blk;

constexpr int kTile = 32;       // keys a wave takes at a time
constexpr int kTerms = 3;       // bf16 terms of a weight
constexpr int kSplitShift = 2;  // log2 of the waves of a workgroup that shares its regions with others
constexpr int kMaxWaves = 8;    // and of any
constexpr int kMaxWgs = 512;    // pieces of the line: 2 for each of the 256 CUs
constexpr int kMinTiles = 8;    // tiles (all waves together) of a piece of the line at least
constexpr int kPartWgs = 256;   // workgroups that take parts of regions: 1 for each CU
constexpr int kMinPart = 4;     // and the tiles of a part at least

struct AttnArgs {
  const uint16_t* q;
  int64_t q_b, q_h;
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  uint32_t page_stride, scale_page_stride;
  int pages, page_shift, heads, D;
  // query heads per KV head; how many of them a region takes (16 or 32, the
  // last one of a KV head fewer), how many regions they make, most rows of one
  int G, qrows, qtiles, rows_max;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int cols, B, Hq, max_len, window;
  float scale_log2e;
  void* out;
  int out_f32;
  float* lse;
  float* ws;
  int line;         // pieces of the line of all tiles; otherwise parts of each region
  int parts_shift;  // log2 of the parts of a region
  int waves_shift;  // log2 of the waves of a workgroup
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The tokens a sequence's new token sees, [lo, n), and the tiles (aligned to
// 32) they lie in.  A sequence that sees nothing counts one tile, which reads
// nothing and puts out the empty row.
struct Span {
  int lo, n, tile0, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int len) {
  Span s;
  s.n = len < 0 ? 0 : (len < a.max_len ? len : a.max_len);
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.tile0 = s.lo / kTile;
  const int end = (s.n + kTile - 1) / kTile;
  s.tiles = end > s.tile0 ? end - s.tile0 : 1;
  return s;
}

// Inclusive sum over the wave's lanes: shifts by 1, 2, 4, 8 inside the rows of
// 16, then each row's last value to the rows behind it.
__device__ __forceinline__ int scan_add(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The work of a launch is the line of all tiles: sequences in order, each
// one's regions (KV head, query tile) in order, each region's tiles in order.
// Every workgroup takes a piece of the line, `per` tiles of it, so the work is
// even whatever the lengths, and the host need not know them.
struct Line {
  int total, per;
  int seq, begin;  // the sequence asked for and where it begins on the line
  Span span;       // and its tokens
};

// BY_TILE: the sequence that holds the first tile of piece x (seq = B if the
// piece lies past the end); otherwise sequence x.
template <bool BY_TILE>
__device__ __forceinline__ Line line_of(const AttnArgs& a, int wgs, int x) {
  const int lane = threadIdx.x & 63, R = a.heads * a.qtiles;
  Line ln;
  ln.seq = a.B;
  ln.begin = 0;
  if (a.B > 64) {
    int sum = 0;
    for (int b = lane; b < a.B; b += 64) sum += span_of(a, a.lens[b]).tiles;
    ln.total = __builtin_amdgcn_readlane(scan_add(sum * R), 63);
  }
  int base = 0, at = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int len = b0 + lane < a.B ? a.lens[b0 + lane] : 0;
    const int v = b0 + lane < a.B ? span_of(a, len).tiles * R : 0;
    const int incl = scan_add(v);
    const int all = __builtin_amdgcn_readlane(incl, 63);
    if (b0 == 0) {
      if (a.B <= 64) ln.total = all;
      const int per = (ln.total + wgs - 1) / wgs;
      ln.per = per > kMinTiles ? per : kMinTiles;
      at = BY_TILE ? x * ln.per : 0;
    }
    const int k = BY_TILE ? (int)__popcll(__ballot(base + incl <= at)) : x - b0;
    if (BY_TILE ? at < base + all : k < 64) {
      ln.seq = uniform(b0 + k);
      ln.begin = base + __builtin_amdgcn_readlane(incl - v, uniform(k));
      ln.span = span_of(a, __builtin_amdgcn_readlane(len, uniform(k)));
      break;
    }
    base += all;
  }
  return ln;
}

// Otherwise each region is cut into 2^parts_shift equal parts, a workgroup each:
// so many tiles to a part, so a short region may have fewer.
__device__ __forceinline__ int part_tiles(const AttnArgs& a, int tiles) {
  const int per = (tiles + (1 << a.parts_shift) - 1) >> a.parts_shift;
  return per > kMinPart ? per : kMinPart;
}

// Floats of a partial result: G rows of D, then G maxima, then G sums.
__host__ __device__ inline int64_t partial_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// Two codes (the low or high half of w) as exact bf16.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if (FMT == 1) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)w, 1.0f, HI));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI));
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// A head's rows in page 0, and how far from there a half tile's (16 keys, all
// in one page) lie.
struct Bases {
  const uint8_t *k, *v;
  const float *ks, *vs;
};
struct Half {
  uint64_t codes, scales;  // bytes and floats from those
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
    const uint8_t* p = at.k + hf[u].codes;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      // pieces past D are read from the row's start and zeroed before use
      const int off = FULL || 64 * c + 16 * g < D ? 64 * c + 16 * g : 0;
      k.c[u][c] = *reinterpret_cast<const u32x4*>(p + (uint32_t)(r * D + off));
    }
    const float* q = at.ks + hf[u].scales;
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
    const uint8_t* p = at.v + hf[u].codes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* x = p + (uint32_t)((4 * g + i) * D + d0);
      if (W == 4) {
        const u32x4 y = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
        for (int w = 0; w < W; ++w) v.c[u][i][w] = y[w];
      } else if (W == 2) {
        const u32x2 y = *reinterpret_cast<const u32x2*>(x);
#pragma unroll
        for (int w = 0; w < W; ++w) v.c[u][i][w] = y[w];
      } else {
        v.c[u][i][0] = *reinterpret_cast<const uint32_t*>(x);
      }
    }
    const float* q = at.vs + hf[u].scales;
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
// The maximum before any score: finite, so that differences of maxima and masked
// scores (-inf) are never NaN; no finite score is below it.
constexpr float kLowest = -3.402823466e38f;

// Maxima without the compiler's canonicalising copies (no operand is a
// signalling NaN); a NaN operand is passed over, as by fmaxf.
__device__ __forceinline__ float max2(float x, float y) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
  return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}

// Over the four lanes that share lane % 16: each swap leaves one row of the
// pair in the first result and the other in the second.
__device__ __forceinline__ float swap_max(float v) {
  typedef unsigned int u2 __attribute__((ext_vector_type(2)));
  const u2 x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = max2(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const u2 y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max2(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

// s = K Q^T with scales, log2 domain, for QT tiles of 16 query heads.
template <int DP, bool FULL, int FMT, int QT>
__device__ __forceinline__ void scores(const AttnArgs& a, const bf16x8 (&qf)[QT][DP / 32], const KeyRegs<DP>& k,
                                       float (&s)[QT][8]) {
  const int g = (threadIdx.x & 63) >> 4;
  typedef uint32_t frag __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    v4f acc[QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) acc[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      u32x4 w = k.c[u][c];
      if (!FULL && 64 * c + 16 * g >= a.D) w = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const frag kf = {widen2<FMT, false>(w[2 * x]), widen2<FMT, true>(w[2 * x]), widen2<FMT, false>(w[2 * x + 1]),
                         widen2<FMT, true>(w[2 * x + 1])};
#pragma unroll
        for (int q = 0; q < QT; ++q)
          acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf), qf[q][2 * c + x], acc[q],
                                                           0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ks = k.s[u][i] * a.scale_log2e;
#pragma unroll
      for (int q = 0; q < QT; ++q) s[q][4 * u + i] = acc[q][i] * ks;
    }
  }
}

// The weights of a tile's scores, the running maximum and sum brought up to
// date.
template <int DP>
__device__ __forceinline__ void weights(float (&s)[8], State<DP>& st) {
  const float mx = swap_max(max2(max3(max3(max3(s[0], s[1], s[2]), s[3], s[4]), s[5], s[6]), s[7]));
  if (__any(mx > st.m)) {
    const float m = max2(st.m, mx);
    const float alpha = __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= alpha;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[j][i] *= alpha;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = __builtin_amdgcn_exp2f(s[i] - st.m);
    st.l += s[i];
  }
}

// O += P V, p the weights times the V scales.
template <int DP, int FMT, int QT>
__device__ __forceinline__ void accumulate(float (&p)[QT][8], const ValueRegs<DP>& v, State<DP> (&st)[QT]) {
  typedef uint32_t frag __attribute__((ext_vector_type(4)));
  // p = sum of kTerms bf16 terms, each the rounded rest of those before
  frag pf[QT][kTerms];
#pragma unroll
  for (int q = 0; q < QT; ++q)
#pragma unroll
    for (int t = 0; t < kTerms; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2 b = {(__bf16)p[q][2 * i], (__bf16)p[q][2 * i + 1]};
        pf[q][t][i] = __builtin_bit_cast(uint32_t, b);
        // (as it is: the low half would be rounded a second time otherwise)
        asm("" : "+v"(pf[q][t][i]));
        p[q][2 * i] -= __uint_as_float(pf[q][t][i] << 16);
        p[q][2 * i + 1] -= __uint_as_float(pf[q][t][i] & 0xffff0000u);
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
      for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
          st[q].o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, vf), __builtin_bit_cast(bf16x8, pf[q][t]), st[q].o[j], 0, 0, 0);
    }
  }
}

// A wave's tiles t, t + waves, ... below `end` (relative to the span's first)
// of one region.  The next tile's keys are loaded as soon as this one's are
// used, its values likewise, so a tile is always in flight.
// The page of each half tile is looked up 32 tiles ahead, one per lane.  Past
// the last token a half may lie anywhere in the cache (ids are clamped): what
// is read there is masked.
template <int DP, bool FULL, int FMT, int QT>
__device__ __forceinline__ void run_tiles(const AttnArgs& a, const Span& sp, int b, int h,
                                          const bf16x8 (&qf)[QT][DP / 32], int t, int end, State<DP> (&st)[QT]) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int ws = a.waves_shift;
  const int32_t* row = a.table + b * a.ld_table;
  const int64_t head_row = (int64_t)h << a.page_shift;
  const Bases at = {a.k_codes + head_row * a.D, a.v_codes + head_row * a.D, a.k_scales + head_row,
                    a.v_scales + head_row};
  const int tile0 = a.window > 0 ? sp.tile0 : 0;
  int ahead = t - (32 << ws);  // the lanes hold where the halves of the 32 tiles from here on lie
  uint64_t codes = 0, scales = 0;

  Half hf[2];
  auto locate = [&](int tt) {
    if (tt - ahead >= (32 << ws)) {
      ahead = tt;
      const uint32_t key = 32 * (uint32_t)(tile0 + tt + ((lane >> 1) << ws)) + 16 * (lane & 1);
      int id = row[min((int)(key >> a.page_shift), a.cols - 1)];
      id = id < 0 ? 0 : (id >= a.pages ? a.pages - 1 : id);
      const uint32_t place = key & ((1u << a.page_shift) - 1);
      codes = (uint64_t)(uint32_t)id * a.page_stride + place * (uint32_t)a.D;
      scales = (uint64_t)(uint32_t)id * a.scale_page_stride + place;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = 2 * ((tt - ahead) >> ws) + u;
      hf[u].codes = lane_value(codes, at);
      hf[u].scales = lane_value(scales, at);
    }
  };

  KeyRegs<DP> k;
  ValueRegs<DP> v;
  // MORE: the next tile's loads go out as this one's registers come free.  A
  // branch around them would make every wait inside the turn wait for all.
  auto turn = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;
    float s[QT][8];
    scores<DP, FULL, FMT, QT>(a, qf, k, s);
    if (MORE) {
      locate(t + (1 << ws));
      load_keys<DP, FULL>(a, at, hf, k);
    }
    const int first = (tile0 + t) * kTile;
    if (first < sp.lo || first + kTile > sp.n) {
      // nothing of a token that is not seen may reach a product
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = first + 16 * u + 4 * g + i;
          const bool seen = j >= sp.lo && j < sp.n;
#pragma unroll
          for (int q = 0; q < QT; ++q) s[q][4 * u + i] = seen ? s[q][4 * u + i] : -__builtin_inff();
          v.s[u][i] = seen ? v.s[u][i] : 0.0f;
#pragma unroll
          for (int w = 0; w < DP / 64; ++w) v.c[u][i][w] = seen ? v.c[u][i][w] : 0u;
        }
    }
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      weights<DP>(s[q], st[q]);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[q][i] *= v.s[i >> 2][i & 3];
    }
    accumulate<DP, FMT, QT>(s, v, st);
    if (MORE) load_values<DP, FULL>(a, at, hf, v);
  };

  if (t >= end) return;
  locate(t);
  load_keys<DP, FULL>(a, at, hf, k);
  load_values<DP, FULL>(a, at, hf, v);
  for (; t + (1 << ws) < end; t += 1 << ws) turn(std::true_type{});
  turn(std::false_type{});
}

// One workgroup takes a piece of the line or a part of one region.  In a piece,
// each region's tiles are dealt to the waves, whose results are joined in LDS; a
// region that lies whole in the workgroup is put out, others go to the
// workspace: of piece w of the line, slot 2w for the region it begins in, slot
// 2w+1 for the one it ends in; of a part, the workgroup's slot.
template <int DP, bool FULL, int FMT, int QT>
__global__ __launch_bounds__(64 * kMaxWaves) void attend_kernel(const AttnArgs a) {
  extern __shared__ float lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int R = a.heads * a.qtiles;
  const int rows_max = a.rows_max;
  constexpr int LD = DP + 4;
  const int waves = 1 << a.waves_shift;
  float* lds_m = lds + waves * rows_max * LD;  // [wave][row]
  float* lds_l = lds_m + waves * rows_max;

  int b, region, tile, left;  // left: tiles of this piece still to do
  Span sp;
  if (a.line) {
    const Line ln = line_of<true>(a, gridDim.x, blockIdx.x);
    b = ln.seq;
    if (b == a.B) return;
    const int at = blockIdx.x * ln.per - ln.begin;
    left = min(ln.per, ln.total - (int)blockIdx.x * ln.per);
    sp = ln.span;
    region = at / sp.tiles;
    tile = at - region * sp.tiles;
  } else {
    const int x = blockIdx.x >> a.parts_shift;
    b = x / R;
    region = x - b * R;
    tile = 0;
    left = 0x7fffffff;
    sp = span_of(a, a.lens[b]);
    if (a.parts_shift > 0) {  // (else the first page is looked up without waiting for the length)
      left = part_tiles(a, sp.tiles);
      tile = (blockIdx.x - (x << a.parts_shift)) * left;
      if (tile >= sp.tiles) return;
    }
  }

  for (;;) {
    const int count = min(sp.tiles - tile, left);
    const int h = a.qtiles == 1 ? region : region / a.qtiles, qt = region - h * a.qtiles;
    const int rows = min(16 * QT, a.G - 16 * QT * qt);
    const int head0 = h * a.G + 16 * QT * qt;
    State<DP> st[QT];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      st[q].m = kLowest;
      st[q].l = 0.0f;
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) st[q].o[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (sp.n > 0) {
      bf16x8 qf[QT][DP / 32];
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const uint16_t* qp = a.q + b * a.q_b + (int64_t)(head0 + 16 * q + c) * a.q_h;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
          const int d = 64 * (j >> 1) + 16 * g + 8 * (j & 1);
          u32x4 w = {0, 0, 0, 0};
          if (16 * q + c < rows && (FULL || d < a.D)) w = *reinterpret_cast<const u32x4*>(qp + d);
          qf[q][j] = __builtin_bit_cast(bf16x8, w);
        }
      }
      run_tiles<DP, FULL, FMT, QT>(a, sp, b, h, qf, tile + wave, tile + count, st);
    }
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      float l = st[q].l;
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      if (16 * q + c < rows) {
        const int at = wave * rows_max + 16 * q + c;
        float* o = lds + at * LD;
#pragma unroll
        for (int j = 0; j < DP / 16; j += 4)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<v4f*>(o + (DP / 16) * (4 * g + i) + j) =
                v4f{st[q].o[j][i], st[q].o[j + 1][i], st[q].o[j + 2][i], st[q].o[j + 3][i]};
        if (g == 0) {
          lds_m[at] = st[q].m;
          lds_l[at] = l;
        }
      }
    }
    __syncthreads();
    const bool whole = count == sp.tiles;
    float* part = nullptr;
    if (!whole) {
      const int64_t slot = a.line ? 2 * (int64_t)blockIdx.x + (tile == 0 ? 1 : 0) : blockIdx.x;
      part = a.ws + slot * partial_floats(rows_max, a.D);
    }
    const int q4 = a.D / 4;
    for (int x = tid; x < rows * q4; x += 64 << a.waves_shift) {
      const int rr = x / q4, d = 4 * (x - rr * q4);
      float m = lds_m[rr];
      for (int w = 1; w < waves; ++w) m = fmaxf(m, lds_m[w * rows_max + rr]);
      float l = 0.0f;
      v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int w = 0; w < waves; ++w) {
        const float f = __builtin_amdgcn_exp2f(lds_m[w * rows_max + rr] - m);
        l = __builtin_fmaf(f, lds_l[w * rows_max + rr], l);
        const v4f ow = *reinterpret_cast<const v4f*>(lds + (w * rows_max + rr) * LD + d);
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
        if (a.lse && d == 0) a.lse[at] = l == 0.0f ? -__builtin_inff() : (m + __log2f(l)) * 0.69314718056f;
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
    if (!a.line || left <= 0) return;
    __syncthreads();  // the next region's results go to the same LDS
    if (++region == R) {
      region = 0;
      ++b;
      sp = span_of(a, a.lens[b]);
    }
  }
}

// Joins the partial results of the regions that several workgroups share.  A
// workgroup takes `rows_wg` rows (query heads; blockIdx.y: which) of a region,
// D/4 threads a row and as many groups of pieces as threads are left.
__global__ __launch_bounds__(256) void join_kernel(const AttnArgs a, int wgs, int rows_wg) {
  __shared__ float lds[256 * 4];
  __shared__ float lds_ml[2][64];
  const int tid = threadIdx.x;
  const int R = a.heads * a.qtiles;
  const int b = blockIdx.x / R, region = blockIdx.x - b * R;
  const int h = a.qtiles == 1 ? region : region / a.qtiles, qt = region - h * a.qtiles;
  const int rows = min(a.qrows, a.G - a.qrows * qt), rows_max = a.rows_max;
  int n;           // of the partial results; number 0 is in slot first, k > 0 in next + k * step
  int64_t first, next, step;
  if (a.line) {
    const Line ln = line_of<false>(a, wgs, b);
    const int t0 = ln.begin + region * ln.span.tiles, t1 = t0 + ln.span.tiles;
    const int w0 = t0 / ln.per;
    n = (t1 - 1) / ln.per - w0 + 1;
    first = 2 * (int64_t)w0 + 1;  // the first of them ends its piece in the region, the others begin theirs
    next = 2 * (int64_t)w0;
    step = 2;
  } else {
    const int tiles = span_of(a, a.lens[b]).tiles, per = part_tiles(a, tiles);
    n = (tiles + per - 1) / per;
    first = next = (int64_t)blockIdx.x << a.parts_shift;
    step = 1;
  }
  if (n == 1) return;  // put out by the workgroup that held it whole

  const int64_t pf = partial_floats(rows_max, a.D);
  const int q4 = a.D / 4, groups = 256 / (q4 * rows_wg);
  const int d = 4 * (tid % q4), rr_wg = tid / q4 % rows_wg, grp = tid / q4 / rows_wg;
  const int rr = blockIdx.y * rows_wg + rr_wg;
  const bool on = grp < groups && rr < rows;
  float m = kLowest, l = 0.0f;
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (on) {
#pragma unroll 4
    for (int k = grp; k < n; k += groups) {
      const float* p = a.ws + (k == 0 ? first : next + k * step) * pf;
      const float pm = p[(int64_t)rows_max * a.D + rr], pl = p[(int64_t)rows_max * a.D + rows_max + rr];
      const v4f po = *reinterpret_cast<const v4f*>(p + (int64_t)rr * a.D + d);
      const float nm = fmaxf(m, pm);
      const float f0 = __builtin_amdgcn_exp2f(m - nm), f1 = __builtin_amdgcn_exp2f(pm - nm);
      m = nm;
      l = l * f0 + pl * f1;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f0 + po[i] * f1;
    }
  }
  if (groups > 1) {
    if (on) {
      *reinterpret_cast<v4f*>(lds + 4 * tid) = o;
      if (d == 0) {
        lds_ml[0][grp * rows_wg + rr_wg] = m;
        lds_ml[1][grp * rows_wg + rr_wg] = l;
      }
    }
    __syncthreads();
    if (!on || grp != 0) return;
    m = kLowest;
    for (int k = 0; k < groups; ++k) m = fmaxf(m, lds_ml[0][k * rows_wg + rr_wg]);
    l = 0.0f;
    o = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < groups; ++k) {
      const float f = __builtin_amdgcn_exp2f(lds_ml[0][k * rows_wg + rr_wg] - m);
      l += f * lds_ml[1][k * rows_wg + rr_wg];
      const v4f ok = *reinterpret_cast<const v4f*>(lds + 4 * (k * rows_wg * q4 + tid));
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += f * ok[i];
    }
  }
  if (!on) return;
  const int64_t at = (int64_t)b * a.Hq + h * a.G + a.qrows * qt + rr;
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
  if (a.lse && d == 0) a.lse[at] = l == 0.0f ? -__builtin_inff() : (m + __log2f(l)) * 0.69314718056f;
}

// ---- host -------------------------------------------------------------------

struct Shape {
  int G, qrows, qtiles, rows;
  int64_t regions, max_len, wgs;  // wgs: pieces of the line; 0: parts of each region
  int waves_shift, parts_shift;
};

static Shape shape_of(const fp8b_kv_cache& c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                      int64_t window) {
  Shape s;
  s.G = (int)(Hq / c.heads);
  // more than 16 heads: two query tiles to a wave, so K and V are read and
  // widened once for both; up to 128 positions, where the registers allow it
  // (32 x 4096 tokens x 4 KV heads, 24 heads each: 45.6 us, 54.4 one tile at a
  // time; 32 x 8192 x 1 KV head of 48, E4M3: 41.9 and 46.7)
  s.qrows = s.G > 16 && c.head_dim <= 128 ? 32 : 16;
  s.qtiles = (s.G + s.qrows - 1) / s.qrows;
  s.rows = s.G < s.qrows ? s.G : s.qrows;
  s.regions = B * c.heads * s.qtiles;
  const int64_t room = cols * c.page_size;
  s.max_len = max_context < room ? max_context : room;
  // the most tiles a region can have: a window reaches into one more
  const int64_t seen = window > 0 && window < s.max_len ? window + kTile - 1 : s.max_len;
  const int64_t tiles = (seen + kTile - 1) / kTile;
  // Three ways to deal out the work (128 positions; tiles: the most of a region).
  //
  // Each region cut into as many equal parts as there are CUs for, and joined by a
  // second launch, which costs about as much as 20 tiles in a row; cut from 24 on
  // (12 of 256 positions, 48 of 64): whole / in parts, 8 regions of 16 tiles 7.0 /
  // 7.9, of 20 7.8 / 7.7, of 24 8.5 / 7.7, of 94 22.6 / 9.4; 64 of 45 13.8 / 11.3; 128
  // of 33 11.8 / 12.6, of 47 14.3 / 14.1.  Half as many parts: 8 of 94 9.7, 64 of 45
  // 12.5; as many workgroups of eight waves 9.3 and 12.1, twice as many of two 10.5 and
  // 11.7.
  const int body = c.head_dim <= 64 ? 64 : (c.head_dim <= 128 ? 128 : 256);
  int parts_shift = 0;
  while ((s.regions << (parts_shift + 1)) <= kPartWgs && (kMinPart << parts_shift) < tiles) ++parts_shift;
  const int64_t saved = tiles - (tiles >> parts_shift);  // in a row, by the parts
  // One workgroup per region while they are short: in a line of all tiles, cut
  // evenly whatever the lengths, a launch costs about 6 us more but no CU waits
  // for the longest region: whole / line, 512 regions of 29 tiles 19.4 / 25.9, of
  // 122 83.6 / 82.8, of 279 177 / 166.
  const int64_t whole = s.regions / 2 < 48 ? 48 : (s.regions / 2 < 128 ? s.regions / 2 : 128);
  s.wgs = 0;
  s.parts_shift = 0;
  if (saved * body > 24 * 128 && tiles <= ((int64_t)64 << parts_shift)) {
    // (in parts / line: 32 regions of 43 tiles 9.6 / 13.1, of 354 19.7 / 22.6; 64 of
    // 178 19.8 / 21.5, of 314, 79 to a part, 33.7 / 33.3)
    s.parts_shift = parts_shift;
    s.waves_shift = kSplitShift;
  } else if (tiles <= whole) {
    // Four waves where 128 or 256 positions fill the body, else eight (64 regions of
    // 23 tiles 4 / 8 waves 8.6 / 9.4, of 256 positions 13.7 / 14.6; 128 of 23 with 80
    // positions 10.7 / 9.9, with 64 8.1 / 7.8), but not more than tiles; fewer where
    // that leaves each only a few tiles and there are regions enough for 12 waves
    // a CU without (2048 regions of 5 tiles: 1 / 2 / 4 / 8 waves 14.6 / 15.7 / 18.4 /
    // 31.1).  Eight waves fill a CU: 272 regions of 33 tiles of 64 positions, E4M3, fp32
    // output, take 26.4 / 16.1 / 11.2 / 10.0 where a third of them is empty, but 26.4 /
    // 20.4 / 13.5 / 16.4 where none is (16 of them wait for the other 256), 512 of them
    // 4 / 8 waves 15.8 / 18.4.
    s.waves_shift = c.head_dim == 128 || c.head_dim == 256 ? 2 : 3;
    while (s.waves_shift > 0 && ((1 << s.waves_shift) > tiles ||
                                 ((5 << s.waves_shift) > tiles && (s.regions << s.waves_shift) > 12 * 256)))
      --s.waves_shift;
  } else {
    // Two workgroups of four waves a CU: 131072 tokens x 8 heads 60.4 us, with four a
    // CU (a fourth of them waits for room) 63.5, with one 58.1; 128 x 6000 x 8 309, 309
    // and 305.  Of two or eight waves 61.6 and 62.9, 311 and 309 (four: 60.1, 305).
    s.waves_shift = kSplitShift;
    const int64_t want = (s.regions * tiles + kMinTiles - 1) / kMinTiles;
    s.wgs = want < kMaxWgs ? want : kMaxWgs;
  }
  return s;
}

int64_t attention_workspace(const fp8b_kv_cache& c, int64_t B, int64_t Hq, int64_t cols, int64_t max_context,
                            int64_t window) {
  const Shape s = shape_of(c, B, Hq, cols, max_context, window);
  const int64_t slots = s.wgs > 0 ? 2 * s.wgs : (s.parts_shift > 0 ? s.regions << s.parts_shift : 0);
  return slots * partial_floats(s.rows, (int)c.head_dim) * (int64_t)sizeof(float);
}

template <int DP, bool FULL, int FMT, int QT>
static int launch_one(const AttnArgs& a, unsigned grid, hipStream_t s) {
  const int waves = 1 << a.waves_shift;
  const size_t lds = (size_t)waves * a.rows_max * (DP + 4 + 2) * sizeof(float);
  hipLaunchKernelGGL((attend_kernel<DP, FULL, FMT, QT>), dim3(grid), dim3(64 * waves), lds, s, a);
  return check_launch();
}
template <int DP, bool FULL, int QT>
static int launch_fmt(const AttnArgs& a, int fmt, unsigned grid, hipStream_t s) {
  return fmt == FP8B_FMT_E5M2 ? launch_one<DP, FULL, 1, QT>(a, grid, s) : launch_one<DP, FULL, 2, QT>(a, grid, s);
}
template <int DP, bool FULL>
static int launch_dp(const AttnArgs& a, int fmt, unsigned grid, hipStream_t s) {
  if (DP <= 128 && a.qrows == 32) return launch_fmt<DP, FULL, DP <= 128 ? 2 : 1>(a, fmt, grid, s);
  return launch_fmt<DP, FULL, 1>(a, fmt, grid, s);
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
  a.page_stride = (uint32_t)c.page_stride;
  a.scale_page_stride = (uint32_t)c.scale_page_stride;
  a.pages = (int)c.pages;
  a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  a.heads = (int)c.heads;
  a.D = (int)c.head_dim;
  a.G = sh.G;
  a.qrows = sh.qrows;
  a.qtiles = sh.qtiles;
  a.rows_max = sh.rows;
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
  a.line = sh.wgs > 0;
  a.parts_shift = sh.parts_shift;
  a.waves_shift = sh.waves_shift;
  a.cols = (int)p.cols;
  const unsigned grid = (unsigned)(sh.wgs > 0 ? sh.wgs : sh.regions << sh.parts_shift);
  int rc;
  // Bodies of 64, 128 and 256 positions; one that D fills asks nothing about D
  // (8 x 1000 tokens x 8 heads 11.4 us, 12.2 by the other; 131072 60.0 and 60.5).  192
  // positions go through the 256 body (32 x 4096 x 8 heads 90.6 us, 256 positions
  // 117): a body of their own spills about 100 registers.
  if (a.D == 64) rc = launch_dp<64, true>(a, c.fmt, grid, s);
  else if (a.D < 64) rc = launch_dp<64, false>(a, c.fmt, grid, s);
  else if (a.D == 128) rc = launch_dp<128, true>(a, c.fmt, grid, s);
  else if (a.D < 128) rc = launch_dp<128, false>(a, c.fmt, grid, s);
  else if (a.D == 256) rc = launch_dp<256, true>(a, c.fmt, grid, s);
  else rc = launch_dp<256, false>(a, c.fmt, grid, s);
  if (rc != FP8B_OK || (!a.line && a.parts_shift == 0)) return rc;
  // Few pieces to a region: its rows side by side in a workgroup (128 x 6000 x 8
  // heads 306 us, 318 with a row each).  Many: one row, the threads shared out
  // over the pieces (131072 x 8 heads 60.3 us, 69.9 with the rows side by side).
  const int fit = 256 / (a.D / 4);
  const int rows_wg = grid <= 4 * sh.regions ? (sh.rows < fit ? sh.rows : fit) : 1;
  const dim3 jgrid((unsigned)sh.regions, (unsigned)((sh.rows + rows_wg - 1) / rows_wg));
  hipLaunchKernelGGL(join_kernel, jgrid, dim3(256), 0, s, a, (int)grid, rows_wg);
  return check_launch();
}

}  // namespace fp8attn

// int8_gemm.hip -- products of 8-bit integer codes with one scale per token and
// one per output channel, dense and per expert.
//
//   y[m][n] = fp32(sum_k a[m][k] w[n][k]) * sa[m] * sw[n] (+ bias[n])
//
// The sum is taken in 32-bit integers by v_mfma_i32_16x16x64_i8, exactly and
// in any order, so a product may be split over waves wherever that is fast.
// The weight rows are the MFMA's first operand, so that a lane's four results
// are four columns of one token.  A weight fragment (16 rows, 64 codes) is one
// packed chunk of 1 KB, 16 bytes a lane; the activations' fragment is 16 bytes
// of 16 rows.
//
// Streaming kernel, for up to 32 rows, which are bound by the weights' bytes
// (16 at a time in grouped products of few tiles, however many there are): a
// workgroup has P panels of 16 weight rows and up to 16 MI tokens; its eight
// waves take every eighth chunk of K, both operands straight to registers, and
// add their sums in LDS.  32 x 8192 -> 28672 takes 38.8 us, 6.1 TB/s of weights.
//
// Tiles, for more rows: four waves have all rows of the tile and a quarter of
// its columns each.  The activations, which all four need, go through LDS, in
// four stages of 128 codes asked for three steps ahead; the weights, which no
// other wave of the workgroup needs, go to registers, two steps ahead, and the
// loads of a chunk are issued behind its last product.  4096 x 7168 -> 18432
// takes 413 us, 2620 TOPS: the matrix units are busy 74% of the time at the
// 1.6 GHz that the power limit leaves; without any load it would take 307 us,
// without stores 375.
//
// Grouped products take pieces of one expert's rows in either way.
#include <algorithm>
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::bf16x2;
using fp8blk::f32_to_bf16_bits;
using fp8blk::u32x2;
using fp8blk::u32x4;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i mfma(v4i w, v4i x, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
}

// How y can be written, by its address and leading dimension: one value at a
// time, four (8 bytes of bf16, 16 of fp32), or 16 bytes of either.
enum class Stores { values, fours, lines };

// A scale as m * 2^e, 1/2 <= |m| < 1 (or m is 0, infinite or NaN).  The product of
// two scales may leave fp32's range where the value that they scale does not;
// that of their m cannot, and the powers of two are exact.
// (With the scales as they are 4096 x 7168 -> 18432 took 397 us against 398, 4096
// x 512 -> 8192 28.7 against 28.8, 64 x 7168 -> 2048 8.30 against 8.35.)
struct Scale {
  float m;
  int e;
};
__device__ __forceinline__ Scale split(float s) {
  return {__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}

// The scales and biases of four columns n .. n+3 (those past the last are the
// last one's).
struct Four {
  Scale scale[4];
  float bias[4];
};
__device__ __forceinline__ Four four(const float* __restrict__ sw, const float* __restrict__ bias, int64_t n, int64_t N) {
  Four f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = min(n + i, N - 1);
    f.scale[i] = split(sw[c]);
    f.bias[i] = bias ? bias[c] : 0.0f;
  }
  return f;
}
// One column's value from its sum.  (Without a bias nothing is added: -0 stays.)
__device__ __forceinline__ float finish(int sum, Scale sa, Scale sw, float bias, bool biased) {
  // (the powers of two last: taken by the sum, which would save a rounding with a
  // bias, they would make NaN of a scale of zero beside a large one)
  const float v = __builtin_amdgcn_ldexpf((float)sum * (sa.m * sw.m), sa.e + sw.e);
  return biased ? v + bias : v;
}

// Four columns n .. n+3 of row y (those below N), from their sums.
template <bool BF16>
__device__ __forceinline__ void store4(const Product& p, int64_t row, int64_t n, const v4i acc, Scale sa, const Four& f,
                                       Stores store) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = finish(acc[i], sa, f.scale[i], f.bias[i], p.bias != nullptr);
  const bool whole = store != Stores::values && n + 4 <= p.N;
  if constexpr (BF16) {
    uint16_t* y = static_cast<uint16_t*>(p.y.p) + row + n;
    if (whole) {
      *reinterpret_cast<u32x2*>(y) = u32x2{f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                                           f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) y[i] = (uint16_t)f32_to_bf16_bits(v[i]);
    }
  } else {
    float* y = static_cast<float*>(p.y.p) + row + n;
    if (whole) {
      *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) y[i] = v[i];
    }
  }
}

// Rows m0 .. m0 + rows - 1 of a product, of one expert or of all.
struct Rows {
  const int32_t* index;  // token of row m, or NULL: row m itself
  int64_t T;             // rows of a
  int64_t m0;
  int rows;
  const int8_t* w;       // packed weights
  const float* sw;
  __device__ __forceinline__ int64_t token(int i) const {
    const int64_t m = m0 + min(i, rows - 1);
    const int64_t t = index ? index[m] : m;
    return t < 0 ? 0 : t < T ? t : T - 1;
  }
};

constexpr int kStreamThreads = 512, kStreamWaves = 8;

__device__ __forceinline__ v4i load_once(const int8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
}

// sums: MI * P KB of LDS.
template <int MI, int P, bool BF16>
__device__ __forceinline__ void stream_tile(const Product& p, const Rows& r, int64_t panel0, Stores store, int* sums) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15,
            g = lane >> 4;
  const int64_t panels = (p.N + 15) / 16;
  const int chunks = (int)((p.K + 127) / 128) * 2;
  const int8_t* ap[MI];
  uint32_t woff[P];
#pragma unroll
  for (int i = 0; i < MI; ++i) ap[i] = p.a + r.token(16 * i + l16) * p.lda + 16 * g;
#pragma unroll
  for (int j = 0; j < P; ++j) woff[j] = (uint32_t)(min(panel0 + j, panels - 1) * 1024) + 16 * lane;
  for (int i = threadIdx.x; i < MI * P * 256; i += kStreamThreads) sums[i] = 0;
  // what the wave's first part of the output needs is asked for before the
  // products (a small one's time is that of a few loads that wait for another)
  auto scales_of = [&](int f) { return four(r.sw, p.bias, (panel0 + f % P) * 16 + 4 * g, p.N); };
  auto row_scale = [&](int f) { return split(p.sa[r.token(16 * (f / P) + l16)]); };
  Four scales = scales_of(min(wave, MI * P - 1));
  Scale sa = row_scale(min(wave, MI * P - 1));
  v4i acc[MI][P];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  // a ring of U chunks in flight; a chunk past the wave's last reads that one
  // again, and is not multiplied
  constexpr int U = P == 1 ? 3 : 2;
  v4i x[U][MI], w[U][P];
  auto fetch = [&](int u, int c) {
    c = min(c, chunks - 1);
    const int8_t* base = r.w + (int64_t)c * panels * 1024;
#pragma unroll
    for (int j = 0; j < P; ++j) w[u][j] = load_once(base + woff[j]);
#pragma unroll
    for (int i = 0; i < MI; ++i) x[u][i] = *reinterpret_cast<const v4i*>(ap[i] + (int64_t)c * 64);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(u, wave + u * kStreamWaves);
  const int mine = (chunks - wave + kStreamWaves - 1) / kStreamWaves;  // chunks of this wave
  int c = wave, n = 0;
  for (; n + U <= mine; n += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) acc[i][j] = mfma(w[u][j], x[u][i], acc[i][j]);
      fetch(u, c + (u + U) * kStreamWaves);
    }
    c += U * kStreamWaves;
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (n + u < mine) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) acc[i][j] = mfma(w[u][j], x[u][i], acc[i][j]);
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) atomicAdd(&sums[((i * P + j) * 4 + q) * 64 + lane], acc[i][j][q]);
  __syncthreads();
  for (int f = wave; f < MI * P; f += kStreamWaves) {
    const int i = f / P, j = f % P;
    const int m = 16 * i + l16;
    const int64_t n = (panel0 + j) * 16 + 4 * g;
    if (m < r.rows && n < p.N) {
      v4i v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = sums[(f * 4 + q) * 64 + lane];
      store4<BF16>(p, (r.m0 + m) * p.y.ld, n, v, sa, scales, store);
    }
    if (f + kStreamWaves < MI * P) {
      scales = scales_of(f + kStreamWaves);
      sa = row_scale(f + kStreamWaves);
    }
  }
}

template <int MI, int P, bool BF16>
__global__ __launch_bounds__(kStreamThreads) void stream_kernel(Product p, int64_t M, Stores store) {
  __shared__ int sums[MI * P * 256];
  const Rows r{nullptr, M, 0, (int)M, p.w, p.sw};
  stream_tile<MI, P, BF16>(p, r, (int64_t)blockIdx.x * P, store, sums);
}

// What a workgroup of a grouped product has: rows of one expert.
struct Item {
  int expert, first, rows;
};

// Inclusive sum over a wave: within rows of 16 lanes, then the rows' last lanes
// to the rows behind them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  return dpp_add<0x143, 0xC>(v);
}

// Rows of expert e, whatever offsets holds.
__device__ __forceinline__ int2 rows_of(const int32_t* __restrict__ offsets, int e, int64_t R) {
  const int lo = max(0, min(offsets[e], (int)R));
  return make_int2(lo, max(lo, min(offsets[e + 1], (int)R)) - lo);
}

// Piece `at` of BM rows or fewer, counted over the experts in turn; false past
// the last.  Every thread of a workgroup of THREADS calls it.
template <int BM, int THREADS>
__device__ __forceinline__ bool find_item(const int32_t* __restrict__ offsets, int E, int64_t R, int at, Item& item) {
  constexpr int kW = THREADS / 64;
  static_assert(1024 <= 2 * THREADS, "the two turns' sums are not written again");
  __shared__ int sum[2][kW];
  __shared__ Item found;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int base = 0, turn = 0;
  for (int e0 = 0; e0 < E && base <= at; e0 += THREADS, turn ^= 1) {
    const int e = e0 + tid;
    const int2 rows = e < E ? rows_of(offsets, e, R) : make_int2(0, 0);
    const int mine = (rows.y + BM - 1) / BM, scan = wave_scan(mine);
    if (lane == 63) sum[turn][w] = scan;
    __syncthreads();
    int earlier = base;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      earlier += i < w ? sum[turn][i] : 0;
      base += sum[turn][i];
    }
    const int in = at - (earlier + scan - mine);
    if (in >= 0 && in < mine) found = Item{e, rows.x + in * BM, min(BM, rows.y - in * BM)};
  }
  if (base <= at) return false;  // the same in every thread
  __syncthreads();
  // the same in every lane, which addresses in scalar registers have to be
  item.expert = __builtin_amdgcn_readfirstlane(found.expert);
  item.first = __builtin_amdgcn_readfirstlane(found.first);
  item.rows = __builtin_amdgcn_readfirstlane(found.rows);
  return true;
}

__device__ __forceinline__ Rows item_rows(const Product& p, const Item& it, int64_t T, const int32_t* index) {
  const int64_t bytes = (p.N + 15) / 16 * 16 * ((p.K + 127) / 128 * 128);
  return Rows{index, T, it.first, it.rows, p.w + it.expert * bytes, p.sw + (int64_t)it.expert * p.N};
}

template <int MI, int P, bool BF16>
__global__ __launch_bounds__(kStreamThreads) void grouped_stream_kernel(Product p, int64_t T,
                                                                        const int32_t* __restrict__ index,
                                                                        const int32_t* __restrict__ offsets, int64_t R,
                                                                        int E, int tiles_n, Stores store) {
  __shared__ int sums[MI * P * 256];
  Item it;
  if (!find_item<16 * MI, kStreamThreads>(offsets, E, R, blockIdx.x / tiles_n, it)) return;
  stream_tile<MI, P, BF16>(p, item_rows(p, it, T, index), (int64_t)(blockIdx.x % tiles_n) * P, store, sums);
}

// ---- tiles ------------------------------------------------------------------

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

constexpr int kStep = 128;  // codes of K a step

// LDS byte of 16-byte chunk `ch` (0 .. 7) of row r of a tile of 128-byte rows;
// chunks are swapped by bits 1-3 of the row, which keeps the fragment reads
// free of bank conflicts.
__device__ __forceinline__ int lds_at(int r, int ch) { return r * kStep + ((ch ^ ((r >> 1) & 7)) << 4); }

// All but the last N loads from memory have arrived, and all reads of LDS.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
}

// A raw buffer over the 4 GiB from base.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)0xFFFFFFFFu, 0x00020000);
}
template <bool ONCE>
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, ONCE ? 2 : 0);  // 2: non-temporal
  return v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}
// 16 bytes a lane from memory to 1 KB of LDS, not through registers.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step_off, int8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, step_off, 0, 0);
}

// G groups of four waves, each with all 16 MI rows of a and 16 NJ of the weights;
// a group takes every G-th step of K.
template <int MI_, int NJ_, int G_ = 1>
struct Cfg {
  static constexpr int MI = MI_, NJ = NJ_, G = G_;
  static constexpr int kWaves = 4, kThreads = 64 * kWaves * G;
  static constexpr int kStage = 16 * MI * kStep * G;  // bytes of LDS
  static constexpr int kRows = 16 * MI, kCols = 64 * NJ;
  static constexpr int kA = kRows / 8 / kWaves;  // pieces of 8 rows of a that a wave brings in a step
  static_assert(kRows % (8 * kWaves) == 0, "pieces split evenly");
};

// The upper half (odd rows of 16 lanes) of a changes places with the lower half
// (even rows) of b.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// The codes of a wave's weight rows in one step.
template <int NJ>
struct Weights {
  v4i w[2][NJ];
};

constexpr int kAhead = 2;  // LDS reads ahead of the products: 480 us with 2 to 4 at 4096 x 7168 -> 18432, 512 with 1

// A wave's sums to 16 MI rows of y, columns from panel `first` on.  Lane
// 16 g + l16 has four columns of row l16 of every panel, 8 bytes of bf16; where
// whole pieces are stored the four lanes of a row change places first
// (v_permlane*_swap), so that each has 16 bytes or more in a row and a store
// instruction fills 64 bytes of a line or more.
// `biased`: whether there is a bias, a constant or not.
template <int MI, int NJ, bool BF16, class B>
__device__ __forceinline__ void store_tile(const Product& p, const Rows& r, int64_t first,
                                           const v4i (&acc)[MI][NJ], const Four (&scales)[NJ], const Scale (&rows)[MI],
                                           B biased, Stores how) {
  static_assert(NJ == 1 || NJ == 2 || NJ == 4, "transposed by twos or fours, or not");
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  if (first * 16 >= p.N) return;
  const bool whole = NJ > 1 && how == Stores::lines && (first + NJ) * 16 <= p.N;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = 16 * i + l16;
    const int64_t row = (r.m0 + m) * p.y.ld;
    constexpr int D = BF16 ? 2 : 4;  // dwords of four columns
    uint32_t d[NJ][D];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = finish(acc[i][j][q], rows[i], scales[j].scale[q], scales[j].bias[q], biased);
      if constexpr (BF16) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const bf16x2 two = {(__bf16)v[2 * q], (__bf16)v[2 * q + 1]};
          d[j][q] = __builtin_bit_cast(uint32_t, two);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) d[j][q] = __float_as_uint(v[q]);
      }
    }
    char* y = static_cast<char*>(p.y.p) + (row + first * 16) * (BF16 ? 2 : 4);
    if (whole) {
#pragma unroll
      for (int q = 0; q < D; ++q) {
        if constexpr (NJ == 4) {
          swap32(d[0][q], d[2][q]);
          swap32(d[1][q], d[3][q]);
          swap16(d[0][q], d[1][q]);
          swap16(d[2][q], d[3][q]);
        } else if constexpr (NJ == 2) {
          swap16(d[0][q], d[1][q]);
        }
      }
      // four panels: lane g has panel g, d[j] its columns 4 j ..; two: lane g
      // has columns 8 (g / 2) .. of panel g % 2, d[j] four of them
      const int at = NJ == 4 ? 16 * g : 16 * (g & 1) + 8 * (g >> 1);
      if (m < r.rows) {
        u32x4* to = reinterpret_cast<u32x4*>(y + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int v = 0; v < NJ * D / 4; ++v)
          to[v] = BF16 ? u32x4{d[2 * v][0], d[2 * v][1], d[2 * v + 1][0], d[2 * v + 1][1]}
                       : u32x4{d[v][0], d[v][1], d[v][D - 2], d[v][D - 1]};
      }
    } else if (m < r.rows) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t n = (first + j) * 16 + 4 * g;
        char* to = y + (16 * j + 4 * g) * (BF16 ? 2 : 4);
        if (how != Stores::values && n + 4 <= p.N) {
          if constexpr (BF16)
            *reinterpret_cast<u32x2*>(to) = u32x2{d[j][0], d[j][1]};
          else
            *reinterpret_cast<u32x4*>(to) = u32x4{d[j][0], d[j][1], d[j][2], d[j][3]};
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < p.N) {
              if constexpr (BF16)
                reinterpret_cast<uint16_t*>(to)[q] = (uint16_t)(d[j][q / 2] >> (16 * (q & 1)));
              else
                reinterpret_cast<uint32_t*>(to)[q] = d[j][q];
            }
        }
      }
    }
  }
}

// st0 .. st3: the stages, C::kStage bytes of LDS each, arrays of their own (so
// that the compiler can tell which of them a load to LDS writes).
template <class C, bool BF16, bool ONCE = false>
__device__ __forceinline__ void tile(const Product& p, const Rows& r, int64_t panel0, Stores store, int8_t* st0,
                                     int8_t* st1, int8_t* st2, int8_t* st3) {
  constexpr int MI = C::MI, NJ = C::NJ, G = C::G;
  // (made anew in every branch of a kernel with several tiles: what follows
  // from it is not kept in registers that the products need)
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = id & 3, group = G > 1 ? id >> 2 : 0;
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t panels = (p.N + 15) / 16;
  // Step t of the group is step G t + group of K; in the last one some groups
  // may have nothing left: they read what is there and multiply nothing.
  const int all = (int)((p.K + kStep - 1) / kStep), steps = (all + G - 1) / G;
  auto of = [&](int t) { return G > 1 ? min(G * t + group, all - 1) : t; };
  const int8_t* abase = p.a + (r.index ? 0 : r.m0 * p.lda);
  uint32_t aoff[C::kA];
#pragma unroll
  for (int q = 0; q < C::kA; ++q) {
    const int row = 8 * (wave + C::kWaves * q) + (lane >> 3);
    const int64_t t = r.index ? r.token(row) : min(row, r.rows - 1);
    aoff[q] = (uint32_t)(t * p.lda) + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const int64_t first = panel0 + wave * NJ;
  uint32_t woff[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) woff[j] = (uint32_t)(min(first + j, panels - 1) * 1024) + 16 * lane;
  const int64_t chunk = panels * 1024;
  auto load_w = [&](v4i (&w)[NJ], int c) {
    const __amdgpu_buffer_rsrc_t b = buffer_at(r.w + c * chunk);
#pragma unroll
    for (int j = 0; j < NJ; ++j) w[j] = load16<ONCE>(b, woff[j]);
  };
  const __amdgpu_buffer_rsrc_t abuf = buffer_at(abase);
  const int own = group * C::kRows * kStep;
  st0 += own;
  st1 += own;
  st2 += own;
  st3 += own;
  auto issue = [&](int8_t* st, int t) {
#pragma unroll
    for (int q = 0; q < C::kA; ++q)
      load_lds(abuf, aoff[q], (uint32_t)(of(t) * kStep), st + 1024 * (wave + C::kWaves * q));
  };
  // the scales, before the products where there are registers for them (a small
  // product's time is that of a few loads that wait for another)
  constexpr bool kEarly = MI * NJ <= 8;
  Four scales[NJ];
  Scale row_scales[MI];
  auto load_scales = [&] {
#pragma unroll
    for (int j = 0; j < NJ; ++j) scales[j] = four(r.sw, p.bias, (first + j) * 16 + 4 * g, p.N);
#pragma unroll
    for (int i = 0; i < MI; ++i) row_scales[i] = split(p.sa[r.token(16 * i + l16)]);
  };
  if (kEarly) load_scales();
  v4i acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const int x_lo = lds_at(l16, g);
  // Step t multiplies stage t % 4 by the weights of set t % 2: the first
  // chunk's products, then the second's, each chunk's registers loaded again
  // for step t + 2 as soon as its products are issued.
  auto step = [&](int t, const int8_t* cur, Weights<NJ>& w, int8_t* refill, bool more_a, bool more_w, bool full,
                  bool live = true) {
    // this wave's part of stage t is in LDS; what may still fly is younger:
    // the stages of t + 1 and t + 2, the weights from t on
    if (full) wait_loads<4 * NJ + 2 * C::kA>(); else wait_loads<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (more_a) issue(refill, t + 3);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int8_t* x = cur + (h ? x_lo ^ 64 : x_lo);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const v4i v = *reinterpret_cast<const v4i*>(x + 2048 * i);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (live) acc[i][j] = mfma(w.w[h][j], v, acc[i][j]);
      }
      if (more_w) load_w(w.w[h], 2 * of(t + 2) + h);
    }
    // the order of the step's instructions: loads to LDS (0x20), LDS reads
    // (0x100), products (0x8), and the loads of weights behind each chunk
    __builtin_amdgcn_sched_group_barrier(0x020, C::kA, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, NJ, 0);
      if (i + kAhead < 2 * MI) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (more_w && (i == MI - 1 || i == 2 * MI - 1)) __builtin_amdgcn_sched_group_barrier(0x020, NJ, 0);
    }
  };
  Weights<NJ> w0, w1;
  // (the loads of steps that are not there read the last one's again: with a
  // branch the compiler would not know how many loads are in flight at the
  // head of the loop, and wait for all)
  const int last = steps - 1;
  issue(st0, 0);
  issue(st1, min(1, last));
  load_w(w0.w[0], 2 * of(0));
  load_w(w0.w[1], 2 * of(0) + 1);
  issue(st2, min(2, last));
  load_w(w1.w[0], 2 * of(min(1, last)));
  load_w(w1.w[1], 2 * of(min(1, last)) + 1);
  int t = 0;
  for (; t + 7 <= steps; t += 4) {
    step(t, st0, w0, st3, true, true, true);
    step(t + 1, st1, w1, st0, true, true, true);
    step(t + 2, st2, w0, st1, true, true, true);
    step(t + 3, st3, w1, st2, true, true, true);
  }
  // one to six more
  auto tail = [&](int u, const int8_t* cur, Weights<NJ>& w, int8_t* refill) {
    if (u < steps)
      step(u, cur, w, refill, u + 3 < steps, u + 2 < steps, u + 2 < steps, G == 1 || G * u + group < all);
  };
  tail(t, st0, w0, st3);
  tail(t + 1, st1, w1, st0);
  tail(t + 2, st2, w0, st1);
  tail(t + 3, st3, w1, st2);
  tail(t + 4, st0, w0, st3);
  tail(t + 5, st1, w1, st0);
  wait_loads<0>();
  if constexpr (G > 1) {
    // the groups' sums join in LDS, 4 KB of a fragment of all four waves
    constexpr int kIn = C::kStage / 4096;
    static_assert(4 * kIn >= (G - 1) * MI * NJ, "the stages hold them");
    st0 -= own;
    st1 -= own;
    st2 -= own;
    st3 -= own;
    auto at = [&](int f) {
      int8_t* st = f / kIn == 0 ? st0 : f / kIn == 1 ? st1 : f / kIn == 2 ? st2 : st3;
      return reinterpret_cast<v4i*>(st + f % kIn * 4096 + wave * 1024 + 16 * lane);
    };
    __syncthreads();
#pragma unroll
    for (int other = 1; other < G; ++other)
      if (group == other)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) *at(((other - 1) * MI + i) * NJ + j) = acc[i][j];
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int other = 1; other < G; ++other)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] += *at(((other - 1) * MI + i) * NJ + j);
  }
  if (!kEarly) load_scales();
  // (a copy of its own for each: 4096 x 512 -> 8192 28.8 us in bf16 against 31.5,
  // but 56.2 in fp32 against 52.7)
  auto out = [&](auto biased) { store_tile<MI, NJ, BF16>(p, r, first, acc, scales, row_scales, biased, store); };
  if constexpr (!BF16)
    out(p.bias != nullptr);
  else if (p.bias)
    out(std::true_type{});
  else
    out(std::false_type{});
}

// Output tile of workgroup `id`: workgroups go round the 8 XCDs in turn, so
// each XCD gets a run of tiles, in groups of 8 tiles of rows, so that the
// workgroups of an XCD share rows and weights in its L2.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int n = tiles_m * tiles_n;
  if (n % 8 == 0) id = id % 8 * (n / 8) + id / 8;
  constexpr int kGroup = 8;
  const int per = kGroup * tiles_n, group = id / per, first = group * kGroup;
  const int rows = min(tiles_m - first, kGroup), in = id - group * per;
  tm = first + in % rows;
  tn = in / rows;
}

template <class C, bool BF16, int OCC>
__global__ __launch_bounds__(C::kThreads, OCC) void tile_kernel(Product p, int64_t M, int tiles_m, int tiles_n,
                                                                Stores store) {
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * C::kRows;
  const Rows r{nullptr, M, m0, (int)min((int64_t)C::kRows, M - m0), p.w, p.sw};
  __shared__ __attribute__((aligned(16))) int8_t st0[C::kStage];
  __shared__ __attribute__((aligned(16))) int8_t st1[C::kStage];
  __shared__ __attribute__((aligned(16))) int8_t st2[C::kStage];
  __shared__ __attribute__((aligned(16))) int8_t st3[C::kStage];
  tile<C, BF16>(p, r, (int64_t)tn * C::NJ * 4, store, st0, st1, st2, st3);
}

// The pieces of a plan, in LDS: experts' rows cut into whole tiles of BM rows
// and last pieces of more than kLittle rows (kind 0), and last pieces of up to
// kLittle rows (kind 1), which are bound by their weights.
constexpr int kLittle = 32;
struct Pieces {
  int lo[1025];         // first row of an expert, and the end
  int before[2][1024];  // pieces of a kind before an expert's
  int sum[2][4];
  Item found;
};
template <int BM>
__device__ __forceinline__ int pieces_of(int n, int kind) {
  const int rest = n % BM;
  return kind ? rest > 0 && rest <= kLittle : n / BM + (rest > kLittle);
}
// Every thread of a workgroup of 256; the kinds' numbers.
template <int BM>
__device__ __forceinline__ int2 count_pieces(Pieces& s, const int32_t* __restrict__ offsets, int E, int64_t R) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int e = tid; e <= E; e += 256) s.lo[e] = max(0, min(offsets[e], (int)R));
  __syncthreads();
  int base[2] = {0, 0};
  for (int e0 = 0; e0 < E; e0 += 256) {
    const int e = e0 + tid;
    const int n = e < E ? max(0, s.lo[e + 1] - s.lo[e]) : 0;
    int mine[2], scan[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mine[k] = pieces_of<BM>(n, k);
      scan[k] = wave_scan(mine[k]);
      if (lane == 63) s.sum[k][w] = scan[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int earlier = base[k];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        earlier += i < w ? s.sum[k][i] : 0;
        base[k] += s.sum[k][i];
      }
      if (e < E) s.before[k][e] = earlier + scan[k] - mine[k];
    }
    __syncthreads();
  }
  return make_int2(__builtin_amdgcn_readfirstlane(base[0]), __builtin_amdgcn_readfirstlane(base[1]));
}
// Piece `rank` of a kind.  Every thread of the workgroup.
template <int BM>
__device__ __forceinline__ Item find_piece(Pieces& s, int E, int kind, int rank) {
  for (int e = threadIdx.x; e < E; e += 256) {
    const int n = max(0, s.lo[e + 1] - s.lo[e]), in = rank - s.before[kind][e];
    if (in >= 0 && in < pieces_of<BM>(n, kind)) {
      const int piece = kind ? n / BM : in;
      s.found = Item{e, s.lo[e] + piece * BM, min(BM, n - piece * BM)};
    }
  }
  __syncthreads();
  // the same in every lane, which addresses in scalar registers have to be
  const Item it{__builtin_amdgcn_readfirstlane(s.found.expert), __builtin_amdgcn_readfirstlane(s.found.first),
                __builtin_amdgcn_readfirstlane(s.found.rows)};
  __syncthreads();
  return it;
}

// Workgroups go round the 8 XCDs in turn.  Each XCD takes an eighth of the
// pieces of kind 0 (times the columns, 64 NJ at a time), then an eighth of
// kind 1, in groups of 8 pieces whose products for all columns follow each
// other, so that what runs at a time on an XCD shares rows and weights in its
// L2.  Both kinds at a time on a compute unit were no faster (870 us one after
// the other, 893 mixed; 4096 tokens, 8 of 256 experts by a skewed router,
// 7168 -> 2048): the loads of one wait behind the other's.  Workgroups past
// the last piece end at once.
template <int NJ, bool BF16>
__global__ __launch_bounds__(256, 2) void grouped_tile_kernel(Product p, int64_t T, const int32_t* __restrict__ index,
                                                              const int32_t* __restrict__ offsets, int64_t R, int E,
                                                              int tiles_n, Stores store) {
  using C = Cfg<8, NJ>;
  __shared__ __attribute__((aligned(16))) int8_t st0[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st1[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st2[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st3[C::kRows * kStep];
  __shared__ Pieces pieces;
  const int2 all = count_pieces<C::kRows>(pieces, offsets, E, R);
  const int xcd = blockIdx.x & 7;
  int64_t i = blockIdx.x >> 3;
  const int64_t items0 = (int64_t)all.x * tiles_n, items1 = (int64_t)all.y * tiles_n;
  int64_t begin = items0 * xcd / 8, end = items0 * (xcd + 1) / 8;
  const int kind = i >= end - begin;
  if (kind) {
    i -= end - begin;
    begin = items1 * xcd / 8;
    end = items1 * (xcd + 1) / 8;
  }
  i += begin;
  if (i >= end) return;
  const int64_t per = 8 * (int64_t)tiles_n;
  const int group = (int)(i / per), in = (int)(i - group * per), rows = min(8, (kind ? all.y : all.x) - 8 * group);
  const int tn = in / rows;
  const Item it = find_piece<C::kRows>(pieces, E, kind, 8 * group + in - tn * rows);
  const Rows r = item_rows(p, it, T, index);
  const int64_t panel0 = (int64_t)tn * NJ * 4;
  if (kind)
    tile<Cfg<2, NJ>, BF16, true>(p, r, panel0, store, st0, st1, st2, st3);
  else if (it.rows <= 64)
    tile<Cfg<4, NJ>, BF16>(p, r, panel0, store, st0, st1, st2, st3);
  else
    tile<C, BF16>(p, r, panel0, store, st0, st1, st2, st3);
}

Stores stores_of(const Mat& y) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(y.p);
  if (p % 16 == 0 && y.ld % (y.bf16 ? 8 : 4) == 0) return Stores::lines;
  return p % (y.bf16 ? 8 : 16) == 0 && y.ld % 4 == 0 ? Stores::fours : Stores::values;
}

template <class C, int OCC>
int launch_tiles(const Product& p, int64_t M, hipStream_t s) {
  const int64_t tiles_m = (M + C::kRows - 1) / C::kRows, tiles_n = (p.N + C::kCols - 1) / C::kCols;
  auto go = [&](auto b) {  // (M N <= 2^36: at most 2^22 tiles)
    hipLaunchKernelGGL((tile_kernel<C, decltype(b)::value, OCC>), dim3((unsigned)(tiles_m * tiles_n)), dim3(C::kThreads),
                       0, s, p, M, (int)tiles_m, (int)tiles_n, stores_of(p.y));
    return check_launch();
  };
  return p.y.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

// Panels of a streaming workgroup: as many as keep the fullest compute unit
// the emptiest, for that many panels there are.
int stream_panels(int64_t panels) {
  constexpr int64_t kUnits = 256;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int P = 1; P <= 8; ++P) {
    const int64_t groups = (panels + P - 1) / P, most = (groups + kUnits - 1) / kUnits * P;
    if (most <= least) {
      least = most;
      best = P;
    }
  }
  return best;
}

int launch_stream(const Product& p, int64_t M, hipStream_t s) {
  const int64_t panels = (p.N + 15) / 16;
  const int P = stream_panels(panels);
  auto go = [&](auto mi, auto pp, auto b) {
    constexpr int MI = decltype(mi)::value, PP = decltype(pp)::value;
    hipLaunchKernelGGL((stream_kernel<MI, PP, decltype(b)::value>), dim3((unsigned)((panels + PP - 1) / PP)),
                       dim3(kStreamThreads), 0, s, p, M, stores_of(p.y));
    return check_launch();
  };
  auto with_type = [&](auto mi, auto pp) {
    return p.y.bf16 ? go(mi, pp, std::true_type{}) : go(mi, pp, std::false_type{});
  };
  auto with_rows = [&](auto pp) {
    if (M <= 16) return with_type(std::integral_constant<int, 1>{}, pp);
    return with_type(std::integral_constant<int, 2>{}, pp);
  };
  switch (P) {
    case 1: return with_rows(std::integral_constant<int, 1>{});
    case 2: return with_rows(std::integral_constant<int, 2>{});
    case 3: return with_rows(std::integral_constant<int, 3>{});
    case 4: return with_rows(std::integral_constant<int, 4>{});
    case 5: return with_rows(std::integral_constant<int, 5>{});
    case 6: return with_rows(std::integral_constant<int, 6>{});
    case 7: return with_rows(std::integral_constant<int, 7>{});
    default: return with_rows(std::integral_constant<int, 8>{});
  }
}

}  // namespace

// Which shape of tiles: the one whose rounds (256 compute units take that many
// tiles at a time) take the least time, by what one round of 7168 columns takes
// in microseconds with many rounds or with one.  Measured (us; 128 x 256,
// 128 x 128, 64 x 128, 32 x 128 and 32 x 64 rows x columns, * for the one chosen):
//   4096 x 7168 -> 18432  413* 505  658  947       1024 x 7168 -> 18432  138* 147  179  279
//    512 x 7168 -> 18432   95   89* 102  141        256 x 7168 -> 18432   54*  65   68   87
//    160 x 7168 -> 18432   48   60   47*  57        128 x 7168 -> 18432   54   39*  50   58
//     64 x 7168 -> 18432   49   33   30*  43   41   256 x 18432 -> 7168  117   82   61*  88
//   2048 x 4096 -> 4096    37*  36   40   55       1024 x 4096 -> 4096    29   21*  22   29
//    512 x 4096 -> 4096    44   19   13*  17        256 x 4096 -> 4096    27   18   11   10*  11
//    128 x 4096 -> 4096    43   18   11    9    8*   64 x 7168 -> 2048         26   16   13   10*
//     64 x 4096 -> 131072 100  106  103* 113        128 x 4096 -> 131072 109* 119  130  171
// A compute unit with one small tile is bound by its loads; from 2048 columns on
// two groups of waves that take the steps in turn are faster (64 x 7168 -> 2048
// 9.6 against 11.2, 128 x 1480 -> 2048 5.0 against 4.5).  That did nothing for
// the larger tiles.
// Up to 16 rows the weights are streamed (16 x 4096 -> 4096 6.3 us, 7.1 by tiles
// of 32 x 64), up to 32 where such tiles would be more than the compute units (32 x
// 7168 -> 18432 25 against 30; 32 x 4096 -> 4096 8.2 against 7.5).
int launch_gemm(const Product& p, int64_t M, hipStream_t s) {
  auto rounds = [&](int64_t rows, int64_t cols) {
    return ((M + rows - 1) / rows * ((p.N + cols - 1) / cols) + 255) / 256;
  };
  const int64_t r21 = rounds(32, 64);
  if (M <= (r21 > 1 ? 32 : 16)) return launch_stream(p, M, s);
  const int64_t t84 = rounds(128, 256) * 43, t82 = rounds(128, 128) * 27, t42 = rounds(64, 128) * 18,
                t22 = rounds(32, 128) * 14, t21 = r21 * 10;
  if (t84 <= std::min({t82, t42, t22, t21})) return launch_tiles<Cfg<8, 4>, 2>(p, M, s);
  if (t82 <= std::min({t42, t22, t21})) return launch_tiles<Cfg<8, 2>, 2>(p, M, s);
  if (t42 <= std::min(t22, t21)) return launch_tiles<Cfg<4, 2>, 3>(p, M, s);
  if (t22 <= t21) return launch_tiles<Cfg<2, 2>, 4>(p, M, s);
  return p.K < 2048 ? launch_tiles<Cfg<2, 1>, 4>(p, M, s) : launch_tiles<Cfg<2, 1, 2>, 4>(p, M, s);
}

int launch_grouped(const Product& p, int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, int E,
                   hipStream_t s) {
  constexpr int NJ = 4, kRows = Cfg<8, NJ>::kRows, kCols = Cfg<8, NJ>::kCols;
  const Stores store = stores_of(p.y);
  // no more pieces than full ones and one begun per expert, nor than rows
  auto pieces = [&](int64_t rows) { return std::min(R, R / rows + E); };
  auto go = [&](auto b) {
    constexpr bool BF16 = decltype(b)::value;
    const int64_t tiles_n = (p.N + kCols - 1) / kCols, tiles = pieces(kRows) * tiles_n;
    // Tiles of 256 columns that would leave compute units without work: panels
    // by two instead, 16 rows at a time (8 tokens, 2 of 8 experts, 7168 -> 2048
    // 18.8 us against 38; from 32 experts on tiles are faster, 47 against 51).
    // Each expert's weights are read again for every 16 of its rows, which the
    // rule does not look at, so it holds for up to about 32 rows an expert (2 of
    // 8 experts, 4096 -> 1792: 64 tokens 18 against 26, 128 25 against 26) and
    // loses beyond (256 tokens 40 against 29, 1024 136 against 36).
    if (tiles < 256) {
      constexpr int MI = 1, P = 2;
      const int64_t columns = (p.N + 16 * P - 1) / (16 * P);
      hipLaunchKernelGGL((grouped_stream_kernel<MI, P, BF16>), dim3((unsigned)(columns * pieces(16 * MI))),
                         dim3(kStreamThreads), 0, s, p, T, row_index, offsets, R, E, (int)columns, store);
    } else {
      // both kinds' shares of an XCD may be one more than an eighth
      hipLaunchKernelGGL((grouped_tile_kernel<NJ, BF16>), dim3((unsigned)((tiles + 7) / 8 * 8 + 16)), dim3(256), 0, s, p,
                         T, row_index, offsets, R, E, (int)tiles_n, store);
    }
    return check_launch();
  };
  return p.y.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace fp8moe

// int8_gemm.hip -- products of 8-bit integer codes with one scale per token and
// one per output channel, dense and per expert.
//
//   y[m][n] = fp32(sum_k a[m][k] w[n][k]) * (sa[m] * sw[n]) (+ bias[n])
//
// The sum is taken in 32-bit integers by v_mfma_i32_16x16x64_i8, exactly and
// in any order, so a product may be split over waves wherever that is fast.
// The weight rows are the MFMA's first operand, so that a lane's four results
// are four columns of one token.  A weight fragment (16 rows, 64 codes) is one
// packed chunk of 1 KB, 16 bytes a lane; the activations' fragment is 16 bytes
// of 16 rows.
//
// Streaming kernel.  A workgroup has P panels of 16 weight rows and up to
// 16 MI tokens; its eight waves take every eighth chunk of K and add their
// sums in LDS.
#include <algorithm>
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::f32_to_bf16_bits;
using fp8blk::u32x2;
using fp8blk::u32x4;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i mfma(v4i w, v4i x, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
}

// Four columns n .. n+3 of row y (those below N), from their sums.
template <bool BF16>
__device__ __forceinline__ void store4(void* y, int64_t row, int64_t n, int64_t N, const v4i acc, float sa,
                                       const float* __restrict__ sw, const float* __restrict__ bias, bool wide) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = min(n + i, N - 1);
    v[i] = (float)acc[i] * (sa * sw[c]);
    if (bias) v[i] += bias[c];
  }
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(y) + row + n;
    if (wide && n + 4 <= N) {
      *reinterpret_cast<u32x2*>(p) = u32x2{f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                                           f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) p[i] = (uint16_t)f32_to_bf16_bits(v[i]);
    }
  } else {
    float* p = static_cast<float*>(y) + row + n;
    if (wide && n + 4 <= N) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) p[i] = v[i];
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

template <int MI, int P, bool BF16>
__device__ __forceinline__ void stream_tile(const Product& p, const Rows& r, int64_t panel0, bool wide) {
  __shared__ int sums[MI * P * 4 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t panels = (p.N + 15) / 16;
  const int chunks = (int)((p.K + 127) / 128) * 2;
  const int8_t* ap[MI];
  const int8_t* wp[P];
#pragma unroll
  for (int i = 0; i < MI; ++i) ap[i] = p.a + r.token(16 * i + l16) * p.lda + 16 * g;
#pragma unroll
  for (int j = 0; j < P; ++j) wp[j] = r.w + min(panel0 + j, panels - 1) * 1024 + 16 * lane;
  v4i acc[MI][P];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  for (int c = wave; c < chunks; c += kStreamWaves) {
    v4i x[MI], w[P];
#pragma unroll
    for (int i = 0; i < MI; ++i) x[i] = *reinterpret_cast<const v4i*>(ap[i] + (int64_t)c * 64);
#pragma unroll
    for (int j = 0; j < P; ++j) w[j] = *reinterpret_cast<const v4i*>(wp[j] + (int64_t)c * panels * 1024);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) acc[i][j] = mfma(w[j], x[i], acc[i][j]);
  }
  for (int i = threadIdx.x; i < MI * P * 256; i += kStreamThreads) sums[i] = 0;
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
      store4<BF16>(p.y.p, (r.m0 + m) * p.y.ld, n, p.N, v, p.sa[r.token(m)], r.sw, p.bias, wide);
    }
  }
}

template <int MI, int P, bool BF16>
__global__ __launch_bounds__(kStreamThreads) void stream_kernel(Product p, int64_t M, int tiles_n, bool wide) {
  const int tn = blockIdx.x % tiles_n;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 16 * MI;
  const Rows r{nullptr, M, m0, (int)min((int64_t)16 * MI, M - m0), p.w, p.sw};
  stream_tile<MI, P, BF16>(p, r, (int64_t)tn * P, wide);
}

// The expert that tile `tile` of BM rows belongs to, counted over the experts
// in turn, and its rows; false past the last one.  Every thread of a workgroup
// of THREADS calls it.
template <int BM, int THREADS>
__device__ __forceinline__ bool find_expert(const int32_t* __restrict__ offsets, int E, int64_t R, int tile, int& expert,
                                            int& first, int& rows) {
  __shared__ int wave_sum[THREADS / 64];
  __shared__ int found[3];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (tid == 0) found[0] = -1;
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + tid;
    int lo = 0, n = 0;
    if (e < E) {
      lo = max(0, min(offsets[e], (int)R));
      n = max(lo, min(offsets[e + 1], (int)R)) - lo;
    }
    const int mine = (n + BM - 1) / BM;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      sum += lane >= d ? o : 0;
    }
    __syncthreads();
    if (lane == 63) wave_sum[w] = sum;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
      before += i < w ? wave_sum[i] : 0;
      all += wave_sum[i];
    }
    const int at = tile - (before + sum - mine);
    if (at >= 0 && at < mine) {
      found[0] = e;
      found[1] = lo + at * BM;
      found[2] = min(BM, n - at * BM);
    }
    base += all;
  }
  __syncthreads();
  expert = found[0];
  first = found[1];
  rows = found[2];
  return expert >= 0;
}

template <int MI, int P, bool BF16>
__global__ __launch_bounds__(kStreamThreads) void grouped_stream_kernel(Product p, int64_t T,
                                                                        const int32_t* __restrict__ index,
                                                                        const int32_t* __restrict__ offsets, int64_t R,
                                                                        int E, int tiles_n, bool wide) {
  int e, first, rows;
  if (!find_expert<16 * MI, kStreamThreads>(offsets, E, R, blockIdx.x / tiles_n, e, first, rows)) return;
  const int64_t bytes = (p.N + 15) / 16 * 16 * ((p.K + 127) / 128 * 128);
  const Rows r{index, T, first, rows, p.w + e * bytes, p.sw + (int64_t)e * p.N};
  stream_tile<MI, P, BF16>(p, r, (int64_t)(blockIdx.x % tiles_n) * P, wide);
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
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}
// 16 bytes a lane from memory to 1 KB of LDS, not through registers.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step_off, int8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, step_off, 0, 0);
}

// WM x 4 waves, each with 16 MI rows of a and 16 NJ of the weights.
template <int MI_, int WM_, int NJ_>
struct Cfg {
  static constexpr int MI = MI_, WM = WM_, NJ = NJ_;
  static constexpr int kWaves = 4 * WM, kThreads = 64 * kWaves;
  static constexpr int kRows = 16 * MI * WM, kCols = 64 * NJ;
  static constexpr int kA = kRows / 8 / kWaves;  // pieces of 8 rows of a that a wave brings in a step
  static_assert(kRows % (8 * kWaves) == 0, "pieces split evenly");
};

// The codes of a wave's weight rows in one step.
template <int NJ>
struct Weights {
  v4i w[2][NJ];
};

#ifndef SGB
#define SGB 2
#endif
template <class C, bool BF16>
__device__ __forceinline__ void tile(const Product& p, const Rows& r, int64_t panel0, bool wide) {
  constexpr int MI = C::MI, NJ = C::NJ;
  __shared__ __attribute__((aligned(16))) int8_t st0[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st1[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st2[C::kRows * kStep];
  __shared__ __attribute__((aligned(16))) int8_t st3[C::kRows * kStep];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 3, wm = wave >> 2;
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t panels = (p.N + 15) / 16;
  const int steps = (int)((p.K + kStep - 1) / kStep);
  const int8_t* abase = p.a + (r.index ? 0 : r.m0 * p.lda);
  uint32_t aoff[C::kA];
#pragma unroll
  for (int q = 0; q < C::kA; ++q) {
    const int row = 8 * (wave + C::kWaves * q) + (lane >> 3);
    const int64_t t = r.index ? r.token(row) : min(row, r.rows - 1);
    aoff[q] = (uint32_t)(t * p.lda) + 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const int64_t first = panel0 + wn * NJ;
  uint32_t woff[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) woff[j] = (uint32_t)(min(first + j, panels - 1) * 1024) + 16 * lane;
  const int64_t chunk = panels * 1024;
  auto load_w = [&](v4i (&w)[NJ], int c) {
    const __amdgpu_buffer_rsrc_t b = buffer_at(r.w + c * chunk);
#pragma unroll
    for (int j = 0; j < NJ; ++j) w[j] = load16(b, woff[j]);
  };
  const __amdgpu_buffer_rsrc_t abuf = buffer_at(abase);
  auto issue = [&](int8_t* st, int t) {
#pragma unroll
    for (int q = 0; q < C::kA; ++q)
      load_lds(abuf, aoff[q], (uint32_t)(t * kStep), st + 1024 * (wave + C::kWaves * q));
  };
  v4i acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const int x_lo = lds_at(16 * MI * wm + l16, g);
  // Step t multiplies stage t % 4 by the weights of set t % 2: the first
  // chunk's products, then the second's, each chunk's registers loaded again
  // for step t + 2 as soon as its products are issued.
  auto step = [&](int t, const int8_t* cur, Weights<NJ>& w, int8_t* refill, bool more_a, bool more_w, bool full) {
    // this wave's part of stage t is in LDS; what may still fly is younger:
    // the stages of t + 1 and t + 2, the weights of t and t + 1
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
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(w.w[h][j], v, acc[i][j]);
      }
      if (more_w) load_w(w.w[h], 2 * (t + 2) + h);
    }
    // LDS reads SGB fragments ahead of the products
    if (SGB > 0) {
      __builtin_amdgcn_sched_group_barrier(0x020, C::kA, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, SGB, 0);
#pragma unroll
      for (int i = 0; i < 2 * MI; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, NJ, 0);
        if (i + SGB < 2 * MI) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (more_w && (i == MI - 1 || i == 2 * MI - 1)) __builtin_amdgcn_sched_group_barrier(0x020, NJ, 0);
      }
    }
  };
  Weights<NJ> w0, w1;
  // (the loads of steps that are not there read the last one's again: with a
  // branch the compiler would not know how many loads are in flight at the
  // head of the loop, and wait for all)
  const int last = steps - 1;
  issue(st0, 0);
  issue(st1, min(1, last));
  load_w(w0.w[0], 0);
  load_w(w0.w[1], 1);
  issue(st2, min(2, last));
  load_w(w1.w[0], 2 * min(1, last));
  load_w(w1.w[1], 2 * min(1, last) + 1);
  int t = 0;
  for (; t + 7 <= steps; t += 4) {
    step(t, st0, w0, st3, true, true, true);
    step(t + 1, st1, w1, st0, true, true, true);
    step(t + 2, st2, w0, st1, true, true, true);
    step(t + 3, st3, w1, st2, true, true, true);
  }
  // one to six more
  auto tail = [&](int u, const int8_t* cur, Weights<NJ>& w, int8_t* refill) {
    if (u < steps) step(u, cur, w, refill, u + 3 < steps, u + 2 < steps, u + 2 < steps);
  };
  tail(t, st0, w0, st3);
  tail(t + 1, st1, w1, st0);
  tail(t + 2, st2, w0, st1);
  tail(t + 3, st3, w1, st2);
  tail(t + 4, st0, w0, st3);
  tail(t + 5, st1, w1, st0);
  wait_loads<0>();
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = 16 * (MI * wm + i) + l16;
    if (m >= r.rows) continue;
    const float sa = p.sa[r.token(m)];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t n = (first + j) * 16 + 4 * g;
      if (n < p.N) store4<BF16>(p.y.p, (r.m0 + m) * p.y.ld, n, p.N, acc[i][j], sa, r.sw, p.bias, wide);
    }
  }
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
                                                                bool wide) {
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * C::kRows;
  const Rows r{nullptr, M, m0, (int)min((int64_t)C::kRows, M - m0), p.w, p.sw};
  tile<C, BF16>(p, r, (int64_t)tn * C::NJ * 4, wide);
}

bool wide_rows(const Mat& y) { return reinterpret_cast<uintptr_t>(y.p) % 16 == 0 && y.ld % 4 == 0; }

}  // namespace

template <class C, int OCC>
int launch_tiles(const Product& p, int64_t M, hipStream_t s) {
  const int64_t tiles_m = (M + C::kRows - 1) / C::kRows, tiles_n = (p.N + C::kCols - 1) / C::kCols;
  if (tiles_m * tiles_n > (1 << 22)) return FP8B_EINVAL;
  auto go = [&](auto b) {
    hipLaunchKernelGGL((tile_kernel<C, decltype(b)::value, OCC>), dim3((unsigned)(tiles_m * tiles_n)), dim3(C::kThreads),
                       0, s, p, M, (int)tiles_m, (int)tiles_n, wide_rows(p.y));
    return check_launch();
  };
  return p.y.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

#ifndef BIG
#define BIG Cfg<8, 1, 4>, 2
#endif
int launch_gemm(const Product& p, int64_t M, hipStream_t s) {
  if (M > 128) return launch_tiles<BIG>(p, M, s);
  if (M > 64) return launch_tiles<Cfg<8, 1, 4>, 2>(p, M, s);
  constexpr int MI = 4, P = 4;
  const int64_t tiles_n = (p.N + 16 * P - 1) / (16 * P), tiles = tiles_n * ((M + 16 * MI - 1) / (16 * MI));
  if (tiles > (1 << 22)) return FP8B_EINVAL;
  auto go = [&](auto b) {
    hipLaunchKernelGGL((stream_kernel<MI, P, decltype(b)::value>), dim3((unsigned)tiles), dim3(kStreamThreads), 0, s, p,
                       M, (int)tiles_n, wide_rows(p.y));
    return check_launch();
  };
  return p.y.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

int launch_grouped(const Product& p, int64_t T, const int32_t* row_index, const int32_t* offsets, int64_t R, int E,
                   hipStream_t s) {
  constexpr int MI = 4, P = 4;
  // no more tiles than full ones and one begun per expert, nor than rows
  const int64_t tiles_n = (p.N + 16 * P - 1) / (16 * P), tiles_m = std::min(R, R / (16 * MI) + E);
  const int64_t tiles = tiles_n * tiles_m;
  if (tiles > (1 << 22)) return FP8B_EINVAL;
  auto go = [&](auto b) {
    hipLaunchKernelGGL((grouped_stream_kernel<MI, P, decltype(b)::value>), dim3((unsigned)tiles), dim3(kStreamThreads),
                       0, s, p, T, row_index, offsets, R, E, (int)tiles_n, wide_rows(p.y));
    return check_launch();
  };
  return p.y.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace fp8moe

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

bool wide_rows(const Mat& y) { return reinterpret_cast<uintptr_t>(y.p) % 16 == 0 && y.ld % 4 == 0; }

}  // namespace

int launch_gemm(const Product& p, int64_t M, hipStream_t s) {
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

// rows.hip -- token rows to their experts and back, and both gradients.
//
// Every kernel goes by tokens: a workgroup has one token's slots and a piece
// of its columns, so that a token's own row (x, out, dout) is read or written
// once and each routed row is touched once.  All are bound by memory.  Rows
// are moved 16 bytes at a time where every row starts on 16 bytes and the
// columns fill them, else one value at a time.
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::bf16_bits_to_f32;
using fp8blk::f32_to_bf16_bits;
using fp8blk::u32x2;
using fp8blk::u32x4;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// W values of one type as they lie in memory.
template <bool BF16, int W>
struct Raw {
  static constexpr int kBytes = W * (BF16 ? 2 : 4);
  using Word = std::conditional_t<BF16 && W == 1, uint16_t, uint32_t>;
  static constexpr int kWords = kBytes / (int)sizeof(Word);
  alignas(kBytes % 16 == 0 ? 16 : sizeof(Word)) Word w[kWords];
};
template <bool BF16, int W>
__device__ __forceinline__ Raw<BF16, W> load(const void* p, int64_t i) {
  Raw<BF16, W> r;
  const char* a = static_cast<const char*>(p) + i * (BF16 ? 2 : 4);
  if constexpr (Raw<BF16, W>::kBytes % 16 == 0) {
#pragma unroll
    for (int q = 0; q < Raw<BF16, W>::kBytes / 16; ++q)
      *reinterpret_cast<u32x4*>(r.w + 4 * q) = *reinterpret_cast<const u32x4*>(a + 16 * q);
  } else {
    static_assert(W == 1, "16 bytes or one value");
    r.w[0] = *reinterpret_cast<const typename Raw<BF16, W>::Word*>(a);
  }
  return r;
}
template <bool BF16, int W>
__device__ __forceinline__ void store(void* p, int64_t i, const Raw<BF16, W>& r) {
  char* a = static_cast<char*>(p) + i * (BF16 ? 2 : 4);
  if constexpr (Raw<BF16, W>::kBytes % 16 == 0) {
#pragma unroll
    for (int q = 0; q < Raw<BF16, W>::kBytes / 16; ++q)
      *reinterpret_cast<u32x4*>(a + 16 * q) = *reinterpret_cast<const u32x4*>(r.w + 4 * q);
  } else {
    *reinterpret_cast<typename Raw<BF16, W>::Word*>(a) = r.w[0];
  }
}
template <bool BF16, int W>
__device__ __forceinline__ float value(const Raw<BF16, W>& r, int i) {
  if constexpr (!BF16)
    return __uint_as_float(r.w[i]);
  else if constexpr (W == 1)
    return bf16_bits_to_f32(r.w[0]);
  else
    return i & 1 ? __uint_as_float(r.w[i / 2] & 0xffff0000u) : __uint_as_float(r.w[i / 2] << 16);
}
template <bool BF16, int W>
__device__ __forceinline__ Raw<BF16, W> raw(const float (&v)[W]) {
  Raw<BF16, W> r;
  if constexpr (!BF16) {
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = __float_as_uint(v[i]);
  } else if constexpr (W == 1) {
    r.w[0] = (uint16_t)f32_to_bf16_bits(v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) r.w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
  }
  return r;
}

// The row of a slot, or -1.
__device__ __forceinline__ int64_t row_of(const int32_t* token_rows, int64_t slot, int64_t R) {
  const int64_t r = token_rows[slot];
  return r >= 0 && r < R ? r : -1;
}

template <bool BF16, int W>
__global__ __launch_bounds__(kThreads) void gather_kernel(const void* x, int64_t ld_x, int64_t N,
                                                          const int32_t* __restrict__ token_rows, int k, int64_t R,
                                                          void* rows, int64_t ld_r) {
  const int64_t t = blockIdx.x;
  for (int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * W; c < N; c += (int64_t)gridDim.y * kThreads * W) {
    const Raw<BF16, W> v = load<BF16, W>(x, t * ld_x + c);
    for (int j = 0; j < k; ++j) {
      const int64_t r = row_of(token_rows, t * k + j, R);
      if (r >= 0) store<BF16, W>(rows, r * ld_r + c, v);
    }
  }
}

template <bool YB, bool OB, int W>
__global__ __launch_bounds__(kThreads) void combine_kernel(const void* y, int64_t ld_y, int64_t R, int64_t N,
                                                           const int32_t* __restrict__ token_rows,
                                                           const float* __restrict__ gates, int k, void* out,
                                                           int64_t ld_o) {
  const int64_t t = blockIdx.x;
  for (int64_t c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * W; c < N; c += (int64_t)gridDim.y * kThreads * W) {
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
    // slots in batches whose loads are all issued before the first is used
    constexpr int B = 8;
    for (int j0 = 0; j0 < k; j0 += B) {
      Raw<YB, W> v[B];
      float g[B];
      bool have[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int64_t r = j0 + j < k ? row_of(token_rows, t * k + j0 + j, R) : -1;
        have[j] = r >= 0;
        if (have[j]) {
          g[j] = gates ? gates[t * k + j0 + j] : 1.0f;
          v[j] = load<YB, W>(y, r * ld_y + c);
        }
      }
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (have[j]) {
#pragma unroll
          for (int i = 0; i < W; ++i) acc[i] = __builtin_fmaf(g[j], value<YB, W>(v[j], i), acc[i]);
        }
    }
    store<OB, W>(out, t * ld_o + c, raw<OB, W>(acc));
  }
}

// One workgroup has a token's whole row, so that its sums need no others'.
template <bool YB, bool OB, int W>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const void* dout, int64_t ld_o, const void* y,
                                                                    int64_t ld_y, int64_t R, int64_t N,
                                                                    const int32_t* __restrict__ token_rows,
                                                                    const float* __restrict__ gates, int k, void* dy,
                                                                    int64_t ld_dy, float* __restrict__ dgates) {
  constexpr int B = 8;
  __shared__ float part[kWaves][B];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int j0 = 0; j0 < k; j0 += B) {
    int64_t r[B];
    float g[B], sum[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      r[j] = j0 + j < k ? row_of(token_rows, t * k + j0 + j, R) : -1;
      g[j] = r[j] >= 0 ? gates[t * k + j0 + j] : 0.0f;
      sum[j] = 0.0f;
    }
    for (int64_t c = (int64_t)threadIdx.x * W; c < N; c += kThreads * W) {
      const Raw<OB, W> d = load<OB, W>(dout, t * ld_o + c);
      Raw<YB, W> v[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (r[j] >= 0) v[j] = load<YB, W>(y, r[j] * ld_y + c);
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (r[j] >= 0) {
          float o[W];
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float di = value<OB, W>(d, i);
            o[i] = g[j] * di;
            sum[j] = __builtin_fmaf(di, value<YB, W>(v[j], i), sum[j]);
          }
          store<YB, W>(dy, r[j] * ld_dy + c, raw<YB, W>(o));
        }
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) sum[j] += __shfl_xor(sum[j], m);
      if (lane == 0) part[w][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x < B && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) s += part[i][threadIdx.x];
      dgates[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

bool wide(const Mat& m) { return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % (m.bf16 ? 8 : 4) == 0; }

// Columns in pieces of a workgroup: enough workgroups that few tokens fill the card.
dim3 grid_of(int64_t T, int64_t N, int W) {
  const int64_t pieces = (N + (int64_t)kThreads * W - 1) / ((int64_t)kThreads * W);
  return dim3((unsigned)T, (unsigned)(pieces < 1024 ? pieces : 1024));
}

// f(y is bf16, out is bf16, wide)
template <class F>
int by_type(bool yb, bool ob, bool w, F f) {
  using T = std::true_type;
  using N = std::false_type;
  if (w) return yb ? (ob ? f(T{}, T{}, T{}) : f(T{}, N{}, T{})) : (ob ? f(N{}, T{}, T{}) : f(N{}, N{}, T{}));
  return yb ? (ob ? f(T{}, T{}, N{}) : f(T{}, N{}, N{})) : (ob ? f(N{}, T{}, N{}) : f(N{}, N{}, N{}));
}

}  // namespace

int launch_gather(const Mat& x, int64_t T, int64_t N, const int32_t* token_rows, int k, int64_t R, const Mat& rows,
                  hipStream_t s) {
  const int W = x.bf16 ? 8 : 4;
  const bool w = wide(x) && wide(rows) && N % W == 0;
  return by_type(x.bf16, x.bf16, w, [&](auto b, auto, auto wd) {
    constexpr int kW = wd.value ? (b.value ? 8 : 4) : 1;
    hipLaunchKernelGGL((gather_kernel<b.value, kW>), grid_of(T, N, kW), dim3(kThreads), 0, s, x.p, x.ld, N, token_rows,
                       k, R, rows.p, rows.ld);
    return check_launch();
  });
}

int launch_combine(const Mat& y, int64_t R, int64_t N, const int32_t* token_rows, const float* gates, int64_t T, int k,
                   const Mat& out, hipStream_t s) {
  const bool w = (R == 0 || wide(y)) && wide(out) && N % (y.bf16 || out.bf16 ? 8 : 4) == 0;
  return by_type(y.bf16, out.bf16, w, [&](auto yb, auto ob, auto wd) {
    constexpr int kW = wd.value ? (yb.value || ob.value ? 8 : 4) : 1;
    hipLaunchKernelGGL((combine_kernel<yb.value, ob.value, kW>), grid_of(T, N, kW), dim3(kThreads), 0, s, y.p, y.ld, R,
                       N, token_rows, gates, k, out.p, out.ld);
    return check_launch();
  });
}

int launch_combine_backward(const Mat& dout, const Mat& y, int64_t R, int64_t N, const int32_t* token_rows,
                            const float* gates, int64_t T, int k, const Mat& dy, float* dgates, hipStream_t s) {
  const bool w = (R == 0 || (wide(y) && wide(dy))) && wide(dout) && N % (y.bf16 || dout.bf16 ? 8 : 4) == 0;
  return by_type(y.bf16, dout.bf16, w, [&](auto yb, auto ob, auto wd) {
    constexpr int kW = wd.value ? (yb.value || ob.value ? 8 : 4) : 1;
    hipLaunchKernelGGL((combine_backward_kernel<yb.value, ob.value, kW>), dim3((unsigned)T), dim3(kThreads), 0, s,
                       dout.p, dout.ld, y.p, y.ld, R, N, token_rows, gates, k, dy.p, dy.ld, dgates);
    return check_launch();
  });
}

}  // namespace fp8moe

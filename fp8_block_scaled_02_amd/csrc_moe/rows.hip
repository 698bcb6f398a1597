// rows.hip -- token rows to their experts and back, and both gradients.
//
// Every kernel goes by tokens: a workgroup has one token's slots and all its
// columns, so that a token's own row (x, out, dout) is read or written once,
// each routed row is touched once, and a slot's gradient is summed where it is
// made, in a fixed order.  All are bound by memory.
//
// Rows are reached through buffer descriptors of their own, whose length is
// that of the row, or none where a slot has no row: loads past it give zeros
// and stores past it do nothing, so there is no branch between the loads of a
// token's slots and all of them are in flight together.  16 bytes at a time
// where rows start on 4 bytes, else one value at a time.
#include <algorithm>
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::bf16_bits_to_f32;
using fp8blk::f32_to_bf16_bits;
using fp8blk::u32x4;

namespace {

constexpr int kMaxThreads = 1024, kMaxWaves = kMaxThreads / 64;
constexpr int kMaxSlots = 8;  // slots whose rows are in flight at a time
// Routed rows that do not fit the last-level cache (256 MiB) are read and
// written non-temporally: combining 470 MB 91 us against 105, 268 MB 55 against
// 64, but 67 MB 21 against 18 and 59 MB, which the products before it left
// there, no faster.
constexpr int64_t kCache = (int64_t)1 << 28;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_at(const void* p, int64_t offset, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(p)) + offset, 0, (int)(uint32_t)bytes,
                                           0x00020000);
}

template <bool BF16>
constexpr int kSize = BF16 ? 2 : 4;

// C consecutive values as they lie in memory: 16-byte words, or one value.
template <bool BF16, int C>
struct Raw {
  static constexpr int kWords = C == 1 ? 1 : C * kSize<BF16> / 4;
  uint32_t w[kWords];
};
template <bool BF16, int C, bool NT = false>
__device__ __forceinline__ Raw<BF16, C> load(__amdgpu_buffer_rsrc_t r, int64_t c) {
  Raw<BF16, C> v;
  const uint32_t at = (uint32_t)c * kSize<BF16>;
  if constexpr (C == 1) {
    v.w[0] = BF16 ? (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0)
                  : (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
  } else {
#pragma unroll
    for (int q = 0; q < Raw<BF16, C>::kWords / 4; ++q) {
      const auto u = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * q, 0, NT ? 2 : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[4 * q + i] = u[i];
    }
  }
  return v;
}
template <bool BF16, int C, bool NT = false>
__device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int64_t c, const Raw<BF16, C>& v) {
  const uint32_t at = (uint32_t)c * kSize<BF16>;
  if constexpr (C == 1) {
    if constexpr (BF16)
      __builtin_amdgcn_raw_buffer_store_b16((unsigned short)v.w[0], r, at, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(v.w[0], r, at, 0, 0);
  } else {
#pragma unroll
    for (int q = 0; q < Raw<BF16, C>::kWords / 4; ++q)
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{v.w[4 * q], v.w[4 * q + 1], v.w[4 * q + 2], v.w[4 * q + 3]}, r,
                                             at + 16 * q, 0, NT ? 2 : 0);
  }
}
template <bool BF16, int C>
__device__ __forceinline__ float value(const Raw<BF16, C>& r, int i) {
  if constexpr (!BF16)
    return __uint_as_float(r.w[i]);
  else if constexpr (C == 1)
    return bf16_bits_to_f32(r.w[0]);
  else
    return i & 1 ? __uint_as_float(r.w[i / 2] & 0xffff0000u) : __uint_as_float(r.w[i / 2] << 16);
}
template <bool BF16, int C>
__device__ __forceinline__ Raw<BF16, C> raw(const float (&v)[C]) {
  Raw<BF16, C> r;
  if constexpr (!BF16) {
#pragma unroll
    for (int i = 0; i < C; ++i) r.w[i] = __float_as_uint(v[i]);
  } else if constexpr (C == 1) {
    r.w[0] = f32_to_bf16_bits(v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) r.w[i] = f32_to_bf16_bits(v[2 * i]) | f32_to_bf16_bits(v[2 * i + 1]) << 16;
  }
  return r;
}

// The row of a slot, or -1.
__device__ __forceinline__ int64_t row_of(const int32_t* token_rows, int64_t slot, int64_t R) {
  const int64_t r = token_rows[slot];
  return r >= 0 && r < R ? r : -1;
}

// Columns of a token in pieces of C: f(first column, whole pieces of C) for U
// pieces of a thread at a time, then one column at a time behind the last
// whole piece.  Pieces past the last are past the descriptors' end.
template <int C, int U, class F, class G>
__device__ __forceinline__ void columns(int64_t N, F whole, G single) {
  const int64_t n = N / C, step = (int64_t)blockDim.x;
  for (int64_t v = threadIdx.x; v < n; v += U * step) whole(v * C, step * C);
  if (C > 1)
    for (int64_t c = n * C + threadIdx.x; c < N; c += step) single(c);
}

// Pieces of a thread at a time: two, one where eight of fp32 would not fit the
// registers.
template <bool BF16, int C>
constexpr int kPieces = !BF16 && C == 8 ? 1 : 2;

template <bool BF16, int C, bool NT>
__global__ __launch_bounds__(kMaxThreads) void gather_kernel(const void* x, int64_t ld_x, int64_t N,
                                                             const int32_t* __restrict__ token_rows, int k, int64_t R,
                                                             void* rows, int64_t ld_r) {
  constexpr int S = kSize<BF16>, U = kPieces<BF16, C>;
  const int64_t t = blockIdx.x;
  auto go = [&](auto cc, auto uu, int64_t c, int64_t step) {
    constexpr int CC = decltype(cc)::value, UU = decltype(uu)::value;
    const __amdgpu_buffer_rsrc_t from = row_at(x, t * ld_x * S, N / CC * CC * S);
    Raw<BF16, CC> v[UU];
#pragma unroll
    for (int u = 0; u < UU; ++u) v[u] = load<BF16, CC>(from, c + u * step);
    for (int j = 0; j < k; ++j) {
      const int64_t r = row_of(token_rows, t * k + j, R);
      const __amdgpu_buffer_rsrc_t to = row_at(rows, r * ld_r * S, r >= 0 ? N / CC * CC * S : 0);
#pragma unroll
      for (int u = 0; u < UU; ++u) store<BF16, CC, NT>(to, c + u * step, v[u]);
    }
  };
  using One = std::integral_constant<int, 1>;
  columns<C, U>(
      N, [&](int64_t c, int64_t step) { go(std::integral_constant<int, C>{}, std::integral_constant<int, U>{}, c, step); },
      [&](int64_t c) { go(One{}, One{}, c, 0); });
}

// S: slots whose rows are in flight at a time.
template <bool YB, bool OB, int C, bool NT, int S>
__global__ __launch_bounds__(kMaxThreads) void combine_kernel(const void* y, int64_t ld_y, int64_t R, int64_t N,
                                                              const int32_t* __restrict__ token_rows,
                                                              const float* __restrict__ gates, int k, void* out,
                                                              int64_t ld_o) {
  constexpr int U = kPieces<YB, C>;
  const int64_t t = blockIdx.x;
  auto go = [&](auto cc, auto uu, int64_t c, int64_t step) {
    constexpr int CC = decltype(cc)::value, UU = decltype(uu)::value;
    float acc[UU][CC];
#pragma unroll
    for (int u = 0; u < UU; ++u)
#pragma unroll
      for (int i = 0; i < CC; ++i) acc[u][i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += S) {
      Raw<YB, CC> v[S][UU];
      float g[S];
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int64_t r = j0 + j < k ? row_of(token_rows, t * k + j0 + j, R) : -1;
        g[j] = r < 0 ? 0.0f : gates ? gates[t * k + j0 + j] : 1.0f;
        const __amdgpu_buffer_rsrc_t from = row_at(y, r * ld_y * kSize<YB>, r >= 0 ? N / CC * CC * kSize<YB> : 0);
#pragma unroll
        for (int u = 0; u < UU; ++u) v[j][u] = load<YB, CC, NT>(from, c + u * step);
      }
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int u = 0; u < UU; ++u)
#pragma unroll
          for (int i = 0; i < CC; ++i) acc[u][i] = __builtin_fmaf(g[j], value<YB, CC>(v[j][u], i), acc[u][i]);
    }
    const __amdgpu_buffer_rsrc_t to = row_at(out, t * ld_o * kSize<OB>, N / CC * CC * kSize<OB>);
#pragma unroll
    for (int u = 0; u < UU; ++u) store<OB, CC, NT>(to, c + u * step, raw<OB, CC>(acc[u]));
  };
  using One = std::integral_constant<int, 1>;
  columns<C, U>(
      N, [&](int64_t c, int64_t step) { go(std::integral_constant<int, C>{}, std::integral_constant<int, U>{}, c, step); },
      [&](int64_t c) { go(One{}, One{}, c, 0); });
}

template <bool YB, bool OB, int C, bool NT, int S>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
    const void* dout, int64_t ld_o, const void* y, int64_t ld_y, int64_t R, int64_t N,
    const int32_t* __restrict__ token_rows, const float* __restrict__ gates, int k, void* dy, int64_t ld_dy,
    float* __restrict__ dgates) {
  constexpr int U = kPieces<YB, C>;
  __shared__ float part[kMaxWaves][S];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int j0 = 0; j0 < k; j0 += S) {
    int64_t r[S];
    float g[S], sum[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      r[j] = j0 + j < k ? row_of(token_rows, t * k + j0 + j, R) : -1;
      g[j] = r[j] < 0 ? 0.0f : gates[t * k + j0 + j];
      sum[j] = 0.0f;
    }
    auto go = [&](auto cc, auto uu, int64_t c, int64_t step) {
      constexpr int CC = decltype(cc)::value, UU = decltype(uu)::value;
      const int64_t bytes = N / CC * CC * kSize<YB>;
      const __amdgpu_buffer_rsrc_t grad = row_at(dout, t * ld_o * kSize<OB>, N / CC * CC * kSize<OB>);
      Raw<OB, CC> d[UU];
      Raw<YB, CC> v[S][UU];
#pragma unroll
      for (int u = 0; u < UU; ++u) d[u] = load<OB, CC>(grad, c + u * step);
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int u = 0; u < UU; ++u)
          v[j][u] = load<YB, CC, NT>(row_at(y, r[j] * ld_y * kSize<YB>, r[j] >= 0 ? bytes : 0), c + u * step);
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int u = 0; u < UU; ++u) {
          float o[CC];
#pragma unroll
          for (int i = 0; i < CC; ++i) {
            const float di = value<OB, CC>(d[u], i);
            o[i] = g[j] * di;
            // (a slot without a row has zeros here, whatever dout holds)
            sum[j] = __builtin_fmaf(r[j] >= 0 ? di : 0.0f, value<YB, CC>(v[j][u], i), sum[j]);
          }
          store<YB, CC, NT>(row_at(dy, r[j] * ld_dy * kSize<YB>, r[j] >= 0 ? bytes : 0), c + u * step, raw<YB, CC>(o));
        }
    };
    using One = std::integral_constant<int, 1>;
    columns<C, U>(
        N,
        [&](int64_t c, int64_t step) { go(std::integral_constant<int, C>{}, std::integral_constant<int, U>{}, c, step); },
        [&](int64_t c) { go(One{}, One{}, c, 0); });
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) sum[j] += __shfl_xor(sum[j], m);
      if (lane == 0) part[w][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x < S && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
      for (int i = 0; i < waves; ++i) s += part[i][threadIdx.x];
      dgates[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

bool wide(const Mat& m) {
  return reinterpret_cast<uintptr_t>(m.p) % 4 == 0 && m.ld * (m.bf16 ? 2 : 4) % 4 == 0;
}

// Threads of a token's workgroup: each has two pieces of a row where that fills
// them.  A launch has fewer than 2^32.
unsigned threads_of(int64_t T, int64_t N, int C) {
  const int64_t pieces = (N / C + 1) / 2, most = T < (1 << 22) ? kMaxThreads : kMaxThreads / 4;
  return (unsigned)std::min(most, std::max<int64_t>(64, (pieces + 63) / 64 * 64));
}

// f(y is bf16, out is bf16, columns of a piece, rows past the cache)
template <class F>
int by_type(bool yb, bool ob, bool w, int64_t row_bytes, F f) {
  using T = std::true_type;
  using N = std::false_type;
  auto with = [&](auto y, auto o) {
    constexpr int C = decltype(y)::value || decltype(o)::value ? 8 : 4;
    if (!w) return f(y, o, std::integral_constant<int, 1>{}, N{});
    return row_bytes >= kCache ? f(y, o, std::integral_constant<int, C>{}, T{}) : f(y, o, std::integral_constant<int, C>{}, N{});
  };
  return yb ? (ob ? with(T{}, T{}) : with(T{}, N{})) : (ob ? with(N{}, T{}) : with(N{}, N{}));
}
// f(slots at a time)
template <class F>
int by_slots(int k, F f) {
  if (k <= 2) return f(std::integral_constant<int, 2>{});
  if (k <= 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, kMaxSlots>{});
}
int64_t row_bytes(const Mat& y, int64_t rows, int64_t N) { return rows * N * (y.bf16 ? 2 : 4); }

}  // namespace

int launch_gather(const Mat& x, int64_t T, int64_t N, const int32_t* token_rows, int k, int64_t R, const Mat& rows,
                  hipStream_t s) {
  return by_type(x.bf16, x.bf16, wide(x) && wide(rows), row_bytes(x, T * k, N), [&](auto b, auto, auto c, auto nt) {
    hipLaunchKernelGGL((gather_kernel<b.value, c.value, nt.value>), dim3((unsigned)T), dim3(threads_of(T, N, c.value)), 0, s,
                       x.p, x.ld, N, token_rows, k, R, rows.p, rows.ld);
    return check_launch();
  });
}

int launch_combine(const Mat& y, int64_t R, int64_t N, const int32_t* token_rows, const float* gates, int64_t T, int k,
                   const Mat& out, hipStream_t s) {
  return by_type(y.bf16, out.bf16, wide(y) && wide(out), row_bytes(y, T * k, N), [&](auto yb, auto ob, auto c, auto nt) {
    return by_slots(k, [&](auto S) {
      hipLaunchKernelGGL((combine_kernel<yb.value, ob.value, c.value, nt.value, S.value>), dim3((unsigned)T),
                         dim3(threads_of(T, N, c.value)), 0, s, y.p, y.ld, R, N, token_rows, gates, k, out.p, out.ld);
      return check_launch();
    });
  });
}

int launch_combine_backward(const Mat& dout, const Mat& y, int64_t R, int64_t N, const int32_t* token_rows,
                            const float* gates, int64_t T, int k, const Mat& dy, float* dgates, hipStream_t s) {
  return by_type(y.bf16, dout.bf16, wide(y) && wide(dy) && wide(dout), row_bytes(y, T * k, N),
                 [&](auto yb, auto ob, auto c, auto nt) {
                   return by_slots(k, [&](auto S) {
                     hipLaunchKernelGGL((combine_backward_kernel<yb.value, ob.value, c.value, nt.value, S.value>),
                                        dim3((unsigned)T), dim3(threads_of(T, N, c.value)), 0, s, dout.p, dout.ld, y.p, y.ld,
                                        R, N, token_rows, gates, k, dy.p, dy.ld, dgates);
                     return check_launch();
                   });
                 });
}

}  // namespace fp8moe

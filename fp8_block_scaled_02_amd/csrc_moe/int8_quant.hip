// int8_quant.hip -- codes and scales in 8-bit integers, and the weights'
// packed layout.
//
// int8_quant: one scale per row.  The row is read once and kept in registers
// while its maximum is found (by the bits of the magnitudes, which order like
// the numbers, a NaN above infinity), then divided.  fp32(x / d) is needed
// exactly, since a code changes where it meets a half: with y = fp32(1 / d),
// t = x y and r = x - t d (exact by FMA), t + r y is the correctly rounded
// quotient (Markstein), where the residual stays in the normal range; rows
// whose maximum is below 2^-62 divide.  Bound by memory.
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::BlockDivisor;
using fp8blk::divide_block;
using fp8blk::u32x2;
using fp8blk::u32x4;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
// Values from which rows are read and codes written non-temporally: 4096 x 7168
// 17.4 us against 18.6, 2048 x 8192 11.0 against 12.4; 8 x 8192 4.3 against 4.1.
constexpr int64_t kLarge = (int64_t)1 << 24;

typedef u32x4 u32x4_on_4 __attribute__((aligned(4)));  // rows start on 4 bytes
template <bool NT>
__device__ __forceinline__ u32x4 words(const void* p) {
  const u32x4_on_4* w = static_cast<const u32x4_on_4*>(p);
  return NT ? __builtin_nontemporal_load(w) : *w;
}

// W values of a row of K from column c < K on, as fp32; columns past the last
// are 0.  TAIL: there may be such columns (the branch costs 2 us of 17.5 at
// 4096 x 7168).
template <bool BF16, int W, bool TAIL, bool NT>
__device__ __forceinline__ void load(const void* row, int64_t c, int64_t K, float (&v)[W]) {
  auto one = [&](int64_t at) {
    return BF16 ? fp8blk::bf16_bits_to_f32(static_cast<const uint16_t*>(row)[at]) : static_cast<const float*>(row)[at];
  };
  if constexpr (W == 1) {
    v[0] = one(c);
  } else if (!TAIL || c + W <= K) {
    static_assert(W == 8, "a piece");
    const char* p = static_cast<const char*>(row) + c * (BF16 ? 2 : 4);
    if constexpr (BF16) {
      const u32x4 u = words<NT>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const u32x4 u = words<NT>(p + 16 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * q + i] = __uint_as_float(u[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = c + i < K ? one(c + i) : 0.0f;
  }
}

template <int W, bool TAIL, bool NT>
__device__ __forceinline__ void quantise(const float (&v)[W], const BlockDivisor& b, bool finite, int8_t* out, int64_t c,
                                         int64_t K) {
  float q[W];
  divide_block<W>(v, q, b);
  int n[W];
#pragma unroll
  for (int i = 0; i < W; ++i) n[i] = finite ? (int)rintf(q[i]) : 0;
  if constexpr (W == 1) {
    out[c] = (int8_t)n[0];
  } else if (!TAIL || c + W <= K) {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = (n[4 * h] & 0xff) | (n[4 * h + 1] & 0xff) << 8 | (n[4 * h + 2] & 0xff) << 16 |
             (uint32_t)n[4 * h + 3] << 24;
    if constexpr (NT)
      __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(out + c));
    else
      *reinterpret_cast<u32x2*>(out + c) = o;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (c + i < K) out[c + i] = (int8_t)n[i];
  }
}

// LANES threads to a row (rows of fewer than a workgroup's threads share one);
// the first H pieces of W values a thread stay in registers, longer rows are
// read again.
template <bool BF16, int W, int LANES, int H, bool TAIL, bool NT>
__global__ __launch_bounds__(LANES < kThreads ? kThreads : LANES) void quant_kernel(const void* x, int64_t M, int64_t K,
                                                                                    int64_t ld_x, int8_t* codes,
                                                                                    int64_t ld_c, float* scales) {
  constexpr int kRows = LANES < kThreads ? kThreads / LANES : 1;
  const int lane = threadIdx.x % LANES;
  const int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  if (m >= M) return;  // whole rows of lanes: no barrier follows where a workgroup has several
  const char* row = static_cast<const char*>(x) + m * ld_x * (BF16 ? 2 : 4);
  int8_t* out = codes + m * ld_c;
  const int64_t c0 = (int64_t)lane * W;
  constexpr int64_t kStep = (int64_t)LANES * W;
  float v[H][W];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (c0 + h * kStep < K) {
      load<BF16, W, TAIL, NT>(row, c0 + h * kStep, K, v[h]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[h][i] = 0.0f;
    }
  }
  uint32_t top = 0;
  auto see = [&](const float (&u)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, __float_as_uint(u[i]) & 0x7fffffffu);
  };
#pragma unroll
  for (int h = 0; h < H; ++h) see(v[h]);
  for (int64_t c = c0 + H * kStep; c < K; c += kStep) {
    float u[W];
    load<BF16, W, TAIL, NT>(row, c, K, u);
    see(u);
  }
  top = __float_as_uint(fp8blk::row16_max_nonneg(__uint_as_float(top)));
  if constexpr (LANES >= 64) {
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  }
  if constexpr (LANES > 64) {
    __shared__ uint32_t part[LANES / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) top = max(top, part[i]);
  }
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;
  BlockDivisor b;
  b.d = top == 0 ? 1.0f : finite ? fmaxf(amax / 127.0f, 0x1.0p-126f) : amax / 127.0f;
  b.y = 1.0f / b.d;
  b.fast = amax >= 0x1.0p-62f;
  if (lane == 0) scales[m] = b.d;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (c0 + h * kStep < K) quantise<W, TAIL, NT>(v[h], b, finite, out, c0 + h * kStep, K);
  for (int64_t c = c0 + H * kStep; c < K; c += kStep) {
    float u[W];
    load<BF16, W, TAIL, NT>(row, c, K, u);
    quantise<W, TAIL, NT>(u, b, finite, out, c, K);
  }
}

// One wave per chunk of the packed layout.  A lane's 16 codes are one load where
// rows start on 16 bytes.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void pack_kernel(const int8_t* __restrict__ w, int64_t N, int64_t K, int64_t ld,
                                                        int64_t stride, int64_t panels, int64_t chunks, int64_t G,
                                                        int8_t* __restrict__ out) {
  const int64_t per = panels * chunks;  // chunks of one matrix
  const int lane = threadIdx.x & 63;
  for (int64_t c = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); c < G * per; c += (int64_t)gridDim.x * kWaves) {
    const int64_t g = c / per, in = c - g * per;
    // panels of 16 rows in turn for a run of 8 chunks (512 codes of a row), so
    // that whole lines are read together
    const int64_t run = in / (8 * panels), at = in - run * 8 * panels, wide = min((int64_t)8, chunks - 8 * run);
    const int64_t p = at / wide, kc = 8 * run + at - p * wide;
    const int64_t n = 16 * p + (lane & 15), k0 = 64 * kc + 16 * (lane >> 4);
    const int8_t* row = w + g * stride + n * ld + k0;
    u32x4 v = {0, 0, 0, 0};
    if (n < N) {
      if (WIDE && k0 + 16 <= K) {
        v = *reinterpret_cast<const u32x4*>(row);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (k0 + i < K) v[i / 4] |= (uint32_t)(uint8_t)row[i] << (8 * (i & 3));
      }
    }
    *reinterpret_cast<u32x4*>(out + (g * per + kc * panels + p) * 1024 + 16 * lane) = v;
  }
}

}  // namespace

int launch_quant(const Mat& x, int64_t M, int64_t K, int8_t* codes, int64_t ld_c, float* scales, hipStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(x.p) % 4 == 0 && x.ld * (x.bf16 ? 2 : 4) % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(codes) % 8 == 0 && ld_c % 8 == 0;
  auto go = [&](auto b, auto w, auto lanes, auto h) {
    constexpr int W = decltype(w)::value, LANES = decltype(lanes)::value, H = decltype(h)::value;
    constexpr int kRows = LANES < kThreads ? kThreads / LANES : 1;
    auto kernel = K % W != 0         ? &quant_kernel<decltype(b)::value, W, LANES, H, true, false>
                  : M * K < kLarge ? &quant_kernel<decltype(b)::value, W, LANES, H, false, false>
                                     : &quant_kernel<decltype(b)::value, W, LANES, H, false, true>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((M + kRows - 1) / kRows)), dim3(kRows > 1 ? kThreads : LANES), 0, s, x.p,
                       M, K, x.ld, codes, ld_c, scales);
    return check_launch();
  };
  // Two pieces of a row to a thread, as few threads as that takes: 65536 rows of
  // 128 take 7.3 us with 16 lanes each, 57 with 256; 128 rows of 20000 4.9 us
  // with 1024, 11.6 with 256.
  auto by_length = [&](auto b) {
    using std::integral_constant;
    using W8 = integral_constant<int, 8>;
    using Two = integral_constant<int, 2>;
    if (!wide) return go(b, integral_constant<int, 1>{}, integral_constant<int, 256>{}, integral_constant<int, 8>{});
    if (K <= 16 * 16) return go(b, W8{}, integral_constant<int, 16>{}, Two{});
    if (K <= 64 * 16) return go(b, W8{}, integral_constant<int, 64>{}, Two{});
    // (a launch has fewer than 2^32 threads)
    if (K <= 256 * 16 || M >= 1 << 22) return go(b, W8{}, integral_constant<int, 256>{}, Two{});
    if (K <= 512 * 16) return go(b, W8{}, integral_constant<int, 512>{}, Two{});
    return go(b, W8{}, integral_constant<int, 1024>{}, Two{});
  };
  return x.bf16 ? by_length(std::true_type{}) : by_length(std::false_type{});
}

int launch_pack(const int8_t* w, int64_t G, int64_t N, int64_t K, int64_t ld, int64_t stride, int8_t* out,
                hipStream_t s) {
  const int64_t panels = (N + 15) / 16, chunks = (K + 127) / 128 * 2;
  const int64_t need = (G * panels * chunks + kWaves - 1) / kWaves;
  const bool wide = reinterpret_cast<uintptr_t>(w) % 16 == 0 && ld % 16 == 0 && stride % 16 == 0;
  auto kernel = wide ? &pack_kernel<true> : &pack_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(need < 65536 ? need : 65536)), dim3(kThreads), 0, s, w, N, K, ld, stride,
                     panels, chunks, G, out);
  return check_launch();
}

}  // namespace fp8moe

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

// W values of a row from column c on, as fp32; columns from K on are 0.
template <bool BF16, int W>
__device__ __forceinline__ void load(const void* row, int64_t c, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = BF16 ? fp8blk::bf16_bits_to_f32(static_cast<const uint16_t*>(row)[c]) : static_cast<const float*>(row)[c];
  } else if constexpr (BF16) {
    static_assert(W == 8, "16 bytes");
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  } else {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const float*>(row) + c + 4 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = __uint_as_float(u[i]);
    }
  }
}

template <int W>
__device__ __forceinline__ void quantise(const float (&v)[W], const BlockDivisor& b, bool finite, int8_t* out) {
  float q[W];
  divide_block<W>(v, q, b);
  int c[W];
#pragma unroll
  for (int i = 0; i < W; ++i) c[i] = finite ? (int)rintf(q[i]) : 0;
  if constexpr (W == 1) {
    out[0] = (int8_t)c[0];
  } else {
    u32x2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = (c[4 * h] & 0xff) | (c[4 * h + 1] & 0xff) << 8 | (c[4 * h + 2] & 0xff) << 16 |
             (uint32_t)c[4 * h + 3] << 24;
    *reinterpret_cast<u32x2*>(out) = o;
  }
}

// One workgroup per row; the first H pieces of W values a thread stay in
// registers, longer rows are read again.
template <bool BF16, int W, int H>
__global__ __launch_bounds__(kThreads) void quant_kernel(const void* x, int64_t K, int64_t ld_x, int8_t* codes,
                                                         int64_t ld_c, float* scales) {
  __shared__ uint32_t part[kWaves];
  const int64_t m = blockIdx.x;
  const char* row = static_cast<const char*>(x) + m * ld_x * (BF16 ? 2 : 4);
  int8_t* out = codes + m * ld_c;
  const int64_t c0 = (int64_t)threadIdx.x * W;
  constexpr int64_t kStep = (int64_t)kThreads * W;
  float v[H][W];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (c0 + h * kStep < K) {
      load<BF16, W>(row, c0 + h * kStep, v[h]);
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
    load<BF16, W>(row, c, u);
    see(u);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) top = max(top, part[i]);
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;
  BlockDivisor b;
  b.d = top == 0 ? 1.0f : finite ? fmaxf(amax / 127.0f, 0x1.0p-126f) : amax / 127.0f;
  b.y = 1.0f / b.d;
  b.fast = amax >= 0x1.0p-62f;
  if (threadIdx.x == 0) scales[m] = b.d;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (c0 + h * kStep < K) quantise<W>(v[h], b, finite, out + c0 + h * kStep);
  for (int64_t c = c0 + H * kStep; c < K; c += kStep) {
    float u[W];
    load<BF16, W>(row, c, u);
    quantise<W>(u, b, finite, out + c);
  }
}

// One thread per 16 bytes of the packed layout.
__global__ __launch_bounds__(kThreads) void pack_kernel(const int8_t* __restrict__ w, int64_t N, int64_t K, int64_t ld,
                                                        int64_t stride, int64_t panels, int64_t chunks, int64_t G,
                                                        int8_t* __restrict__ out) {
  const int64_t per = panels * chunks;  // chunks of one matrix
  for (int64_t c = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); c < G * per;
       c += (int64_t)gridDim.x * kWaves) {
    const int64_t g = c / per, in = c - g * per;
    const int64_t kc = in / panels, p = in - kc * panels;
    const int lane = threadIdx.x & 63;
    const int64_t n = 16 * p + (lane & 15), k0 = 64 * kc + 16 * (lane >> 4);
    const int8_t* row = w + g * stride + n * ld + k0;
    uint32_t v[4] = {0, 0, 0, 0};
    if (n < N) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k0 + i < K) v[i / 4] |= (uint32_t)(uint8_t)row[i] << (8 * (i & 3));
    }
    *reinterpret_cast<u32x4*>(out + c * 1024 + 16 * lane) = u32x4{v[0], v[1], v[2], v[3]};
  }
}

}  // namespace

int launch_quant(const Mat& x, int64_t M, int64_t K, int8_t* codes, int64_t ld_c, float* scales, hipStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.ld % (x.bf16 ? 8 : 4) == 0 && K % 8 == 0 &&
                    reinterpret_cast<uintptr_t>(codes) % 8 == 0 && ld_c % 8 == 0;
  auto go = [&](auto b, auto w) {
    constexpr int W = decltype(w)::value;
    constexpr int H = W == 1 ? 8 : 4;
    hipLaunchKernelGGL((quant_kernel<decltype(b)::value, W, H>), dim3((unsigned)M), dim3(kThreads), 0, s, x.p, K, x.ld,
                       codes, ld_c, scales);
    return check_launch();
  };
  using W8 = std::integral_constant<int, 8>;
  using W1 = std::integral_constant<int, 1>;
  if (x.bf16) return wide ? go(std::true_type{}, W8{}) : go(std::true_type{}, W1{});
  return wide ? go(std::false_type{}, W8{}) : go(std::false_type{}, W1{});
}

int launch_pack(const int8_t* w, int64_t G, int64_t N, int64_t K, int64_t ld, int64_t stride, int8_t* out,
                hipStream_t s) {
  const int64_t panels = (N + 15) / 16, chunks = (K + 127) / 128 * 2;
  const int64_t need = (G * panels * chunks + kWaves - 1) / kWaves;
  hipLaunchKernelGGL(pack_kernel, dim3((unsigned)(need < 65536 ? need : 65536)), dim3(kThreads), 0, s, w, N, K, ld,
                     stride, panels, chunks, G, out);
  return check_launch();
}

}  // namespace fp8moe

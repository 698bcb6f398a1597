// route.hip -- the router: each token's experts and weights, the plan that
// sorts (token, slot) pairs by expert, and the weights' gradient.
//
// Choosing.  G lanes hold one token's E logits, V to a lane (lane l those of
// experts l, l + G, ...), as unsigned keys that order like the numbers.  k
// times over, the largest key is found in the lane, then over the G lanes;
// among the lanes that hold it the lowest expert wins, and its key leaves.
// The first one chosen is the maximum that the softmax subtracts, so the
// weights follow from the k chosen (or all E) logits without another pass.
//
// Sorting.  A stable counting sort in two launches (one while the tokens fit
// one workgroup): every workgroup counts its tokens' experts in LDS while it
// chooses them; then each workgroup adds up what comes before it (all rows of
// lower experts, rows of its own expert in earlier workgroups and waves) and
// places its rows.  A wave places 64 slots at a time: lanes with the same
// expert find each other by one ballot per bit of the expert's number, and
// count those before them.  Integers only, so the order is the definition's
// whatever the timing.
#include <algorithm>
#include <type_traits>

#include "../csrc/common.hpp"
#include "moe_launch.hpp"

namespace fp8moe {

using fp8blk::bf16_bits_to_f32;
using fp8blk::f32_to_bf16_bits;

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kMaxE = 1024;
constexpr int kBlockTokens = 32;   // tokens a workgroup chooses for at a time with 16 lanes to each
constexpr int64_t kMaxBlocks = 256;

// ---- reductions over the G lanes of a token ---------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int G, class F>
__device__ __forceinline__ uint32_t reduce(uint32_t v, F f) {
  static_assert(G == 16 || G == 64, "a row of lanes or the wave");
  v = f(v, dpp<0xB1>(v));    // lanes 1 apart,
  v = f(v, dpp<0x4E>(v));    // 2 apart,
  v = f(v, dpp<0x141>(v));   // the half row mirrored,
  v = f(v, dpp<0x140>(v));   // the row mirrored
  if constexpr (G == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t min_of(uint32_t v) {
  return reduce<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ float sum_of(float v) {
  return __uint_as_float(reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Keys that order like the numbers: NaN above all, -0 as 0, -inf (and places
// past the last expert) 0, which is never chosen.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  if (u == 0xFF800000u) return 0;
  return (u >> 31) ? ~u : u | 0x80000000u;
}

template <bool BF16>
__device__ __forceinline__ float load(const void* p, int64_t i) {
  if constexpr (BF16)
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else
    return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store(void* p, int64_t i, float v) {
  if constexpr (BF16)
    static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
  else
    static_cast<float*>(p)[i] = v;
}

// ---- choosing ---------------------------------------------------------------

struct Route {
  const void* logits;
  int64_t ld, T;
  int E, k, renormalize;
  float* gates;
};
struct Sort {
  int64_t T;
  int E, k;
  int64_t per_block;  // tokens of a workgroup
  Plan p;
  int32_t* hist;      // [workgroups][E]
};

// The chosen ones of a token (lanes of the same wave write and read them).
struct Chosen {
  float value[64];
  int expert[64];
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Token t by the G lanes that call it; its experts are counted in `count`.
template <bool BF16, int G, int V>
__device__ __forceinline__ void choose(const Route& r, int64_t t, int32_t* __restrict__ experts, Chosen& c,
                                       int* count) {
  const int l = threadIdx.x % G;
  float x[V];
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = l + i * G < r.E ? load<BF16>(r.logits, t * r.ld + l + i * G) : -__builtin_inff();
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = key_of(x[i]);
  int n = 0;  // experts chosen
  for (; n < r.k; ++n) {
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max(top, key[i]);
    const uint32_t best = max_of<G>(top);
    if (best == 0) break;  // the same in all G lanes
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(l + i * G) : at;
    const uint32_t e = min_of<G>(at);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((uint32_t)(l + i * G) == e) {
        key[i] = 0;
        c.value[n] = x[i];
        c.expert[n] = (int)e;
      }
    }
  }
  wave_sync();
  const float m = n > 0 ? c.value[0] : 0.0f;
  float sum = 0.0f;
  if (r.renormalize) {
    for (int j = l; j < n; j += G) sum += expf(c.value[j] - m);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += expf(x[i] - m);  // -inf adds 0
  }
  sum = sum_of<G>(sum);
  for (int j = l; j < r.k; j += G) {
    const int e = j < n ? c.expert[j] : -1;
    r.gates[t * r.k + j] = j < n ? expf(c.value[j] - m) / sum : 0.0f;
    experts[t * r.k + j] = e;
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  wave_sync();  // c is written again for the next token
}

// ---- placing ----------------------------------------------------------------

struct PlaceLds {
  int count[kWaves][kMaxE];  // rows of an expert in a wave's part, then where the next one goes
  int total[kThreads], before[kThreads];
  int scan[kWaves];
};

// Workgroup b of nb, every thread of it.
__device__ __forceinline__ void place(const Sort& s, int b, int nb, PlaceLds& lds) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, E = s.E;
  const int64_t first = (int64_t)b * s.per_block * s.k;
  const int64_t n = min(s.per_block, s.T - b * s.per_block) * s.k;  // slots of this workgroup
  const int64_t part = (n + kWaves * 64 - 1) / (kWaves * 64) * 64;  // and of a wave
  const int64_t lo = min(n, w * part), hi = min(n, lo + part);
  for (int i = tid; i < kWaves * E; i += kThreads) lds.count[i / E][i % E] = 0;
  __syncthreads();
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const int e = s.p.experts[first + i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&lds.count[w][e], 1);
  }
  __syncthreads();
  // in parts of kThreads experts: all rows of an expert, and those of it before this workgroup
  int64_t base = 0;  // rows of the experts before the part
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    int all = 0, before = 0;
    if (nb > 1) {
      if (e < E) {
#pragma unroll 8
        for (int i = 0; i < nb; ++i) {
          const int h = s.hist[(int64_t)i * E + e];
          all += h;
          before += i < b ? h : 0;
        }
      }
    } else if (e < E) {
#pragma unroll
      for (int i = 0; i < kWaves; ++i) all += lds.count[i][e];
    }
    int sum = all;  // inclusive scan over the wave's experts
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      sum += lane >= d ? o : 0;
    }
    if (lane == 63) lds.scan[w] = sum;
    __syncthreads();
    int earlier = 0, whole = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      earlier += i < w ? lds.scan[i] : 0;
      whole += lds.scan[i];
    }
    const int64_t start = base + earlier + sum - all;
    if (e < E) {
      if (b == 0) s.p.offsets[e] = (int)start;
      int at = (int)start + before;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        const int c = lds.count[i][e];
        lds.count[i][e] = at;
        at += c;
      }
    }
    base += whole;
    __syncthreads();
  }
  if (b == 0 && tid == 0) s.p.offsets[E] = (int)base;
  // rows that no slot has: this workgroup's share
  const int64_t R = s.T * s.k;
  for (int64_t r = base + (int64_t)b * kThreads + tid; r < R; r += (int64_t)nb * kThreads) s.p.row_index[r] = -1;
  const int bits = 32 - __builtin_clz(E);  // E <= 2^bits - 1 tells an empty slot from the experts
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    int e = i < hi ? s.p.experts[first + i] : -1;
    if ((unsigned)e >= (unsigned)E) e = E;
    uint64_t same = ~0ull;
    for (int j = 0; j < bits; ++j) {
      const uint64_t one = __ballot((e >> j) & 1);
      same &= (e >> j) & 1 ? one : ~one;
    }
    const int ahead = __popcll(same & ((1ull << lane) - 1));
    const bool kept = e < E;
    int at = 0;
    if (kept) at = lds.count[w][e] + ahead;
    wave_sync();
    if (kept && (same >> lane) == 1) lds.count[w][e] = at + 1;  // the last lane of its expert
    wave_sync();
    if (i < hi) s.p.token_rows[first + i] = kept ? at : -1;
    if (kept) s.p.row_index[at] = (int)((uint32_t)(first + i) / (uint32_t)s.k);
  }
}

template <bool BF16, int G, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(Route r, Sort s) {
  constexpr int kGroups = kThreads / G;
  __shared__ Chosen chosen[kGroups];
  __shared__ PlaceLds lds;
  int* count = lds.count[0];
  for (int e = threadIdx.x; e < r.E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int g = threadIdx.x / G;
  const int64_t end = min(r.T, (int64_t)(blockIdx.x + 1) * s.per_block);
  // every wave goes round as often as its first token needs: the lanes of a
  // wave stay together, groups past the end repeat the last token
  for (int64_t t0 = (int64_t)blockIdx.x * s.per_block; t0 < end; t0 += kGroups) {
    const int64_t t = t0 + g;
    if (t < end) choose<BF16, G, V>(r, t, s.p.experts, chosen[g], count);
  }
  __syncthreads();
  if (gridDim.x == 1) {
    __threadfence_block();
    place(s, 0, 1, lds);
  } else {
    for (int e = threadIdx.x; e < r.E; e += kThreads) s.hist[(int64_t)blockIdx.x * r.E + e] = count[e];
  }
}

__global__ __launch_bounds__(kThreads) void count_kernel(Sort s) {
  __shared__ int count[kMaxE];
  for (int e = threadIdx.x; e < s.E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * s.per_block, last = min(s.T, first + s.per_block);
  for (int64_t i = first * s.k + threadIdx.x; i < last * s.k; i += kThreads) {
    const int e = s.p.experts[i];
    if ((unsigned)e < (unsigned)s.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < s.E; e += kThreads) s.hist[(int64_t)blockIdx.x * s.E + e] = count[e];
}

__global__ __launch_bounds__(kThreads) void place_kernel(Sort s) {
  __shared__ PlaceLds lds;
  place(s, blockIdx.x, gridDim.x, lds);
}

__global__ __launch_bounds__(kThreads) void no_tokens_kernel(int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += kThreads) offsets[e] = 0;
}

// ---- the weights' gradient --------------------------------------------------

template <bool BF16, int G, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ dgates, const void* logits,
                                                             int64_t ld, const float* __restrict__ gates,
                                                             const int32_t* __restrict__ experts, int64_t T, int E,
                                                             int k, int renormalize, void* dlogits, int64_t ld_d) {
  const int l = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (t >= T) return;
  float x[V], p[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = !renormalize && l + i * G < E ? load<BF16>(logits, t * ld + l + i * G) : -__builtin_inff();
    p[i] = 0.0f;
  }
  float dot = 0.0f;
  for (int j = l; j < k; j += G)
    if ((unsigned)experts[t * k + j] < (unsigned)E) dot += gates[t * k + j] * dgates[t * k + j];
  dot = sum_of<G>(dot);
  if (!renormalize) {
    // the maximum is that of the numbers; a NaN or +inf makes the sum NaN as in the forward pass
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, key_of(x[i]));
    top = max_of<G>(top);
    if (top != 0) {
      const float m = top == 0xFFFFFFFFu ? __builtin_nanf("")
                                         : __uint_as_float(top >> 31 ? top & 0x7FFFFFFFu : ~top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = expf(x[i] - m);
        sum += p[i];
      }
      sum = sum_of<G>(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = -(p[i] / sum) * dot;
    }
  }
  for (int j = 0; j < k; ++j) {
    const int e = experts[t * k + j];
    if ((unsigned)e < (unsigned)E && e % G == l) {
      const float g = gates[t * k + j], dg = dgates[t * k + j];
      const float add = renormalize ? g * (dg - dot) : g * dg;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] += e / G == i ? add : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (l + i * G < E) store<BF16>(dlogits, t * ld_d + l + i * G, p[i]);
}

Sort sort_of(int64_t T, int E, int k, const Plan& p, int32_t* ws) {
  const int64_t blocks = std::max<int64_t>(sort_blocks(T), 1);
  return Sort{T, E, k, (T + blocks - 1) / blocks, p, ws};
}

int no_tokens(int32_t* offsets, int E, hipStream_t s) {
  hipLaunchKernelGGL(no_tokens_kernel, dim3(1), dim3(kThreads), 0, s, offsets, E);
  return check_launch();
}

// f(bool_constant<BF16>, G, V) for rows of E logits.
template <class F>
int by_width(bool bf16, int E, F f) {
  auto with = [&](auto b) {
    using std::integral_constant;
    if (E <= 16) return f(b, integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (E <= 64) return f(b, integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (E <= 128) return f(b, integral_constant<int, 16>{}, integral_constant<int, 8>{});
    if (E <= 256) return f(b, integral_constant<int, 16>{}, integral_constant<int, 16>{});
    return f(b, integral_constant<int, 64>{}, integral_constant<int, 16>{});
  };
  return bf16 ? with(std::true_type{}) : with(std::false_type{});
}

}  // namespace

int64_t sort_blocks(int64_t T) { return std::min((T + kBlockTokens - 1) / kBlockTokens, kMaxBlocks); }

int launch_route(const Mat& logits, int64_t T, int E, int k, bool renormalize, float* gates, const Plan& p, int32_t* ws,
                 hipStream_t s) {
  if (T == 0) return no_tokens(p.offsets, E, s);
  const Sort sort = sort_of(T, E, k, p, ws);
  const unsigned blocks = (unsigned)((T + sort.per_block - 1) / sort.per_block);
  const Route r{logits.p, logits.ld, T, E, k, renormalize, gates};
  int rc = by_width(logits.bf16, E, [&](auto b, auto G, auto V) {
    hipLaunchKernelGGL((route_kernel<b.value, G.value, V.value>), dim3(blocks), dim3(kThreads), 0, s, r, sort);
    return check_launch();
  });
  if (rc != FP8B_OK || blocks == 1) return rc;
  hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kThreads), 0, s, sort);
  return check_launch();
}

int launch_sort(int64_t T, int E, int k, const Plan& p, int32_t* ws, hipStream_t s) {
  if (T == 0) return no_tokens(p.offsets, E, s);
  const Sort sort = sort_of(T, E, k, p, ws);
  const unsigned blocks = (unsigned)((T + sort.per_block - 1) / sort.per_block);
  if (blocks > 1) {
    hipLaunchKernelGGL(count_kernel, dim3(blocks), dim3(kThreads), 0, s, sort);
    if (const int rc = check_launch()) return rc;
  }
  hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kThreads), 0, s, sort);
  return check_launch();
}

int launch_route_backward(const float* dgates, const Mat& logits, const float* gates, const int32_t* experts, int64_t T,
                          int E, int k, bool renormalize, const Mat& dlogits, hipStream_t s) {
  return by_width(dlogits.bf16, E, [&](auto b, auto G, auto V) {
    const unsigned blocks = (unsigned)((T + 256 / G.value - 1) / (256 / G.value));
    hipLaunchKernelGGL((route_backward_kernel<b.value, G.value, V.value>), dim3(blocks), dim3(256), 0, s, dgates,
                       logits.p, logits.ld, gates, experts, T, E, k, (int)renormalize, dlogits.p, dlogits.ld);
    return check_launch();
  });
}

}  // namespace fp8moe

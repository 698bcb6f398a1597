// route.hip -- the router: each token's experts and weights, the plan that
// sorts (token, slot) pairs by expert, and the weights' gradient.
//
// Choosing.  G lanes hold one token's E logits, V to a lane (lane l those of
// experts l, l + G, ...), as unsigned keys that order like the numbers.  The
// k-th largest of 16 lanes' largest keys (of 16 sets of four lanes' in a whole
// wave) is a lower bound of the token's k-th largest key; what reaches it,
// rarely much more than k, goes to LDS, where every candidate counts those
// before it (larger, or equal and of a lower expert): that is its slot.  Where
// that does not hold (k > 16, more than 64 candidates), k times over the largest
// key is found in the lane, then over the lanes, and leaves.  For 16384 tokens, 8
// of 256 experts, the k-fold search took 14.4 us, this 9.4: half of that is
// vector instructions (2770 a SIMD of 4 cycles each), the rest a workgroup's
// chain of loads and LDS, of which a compute unit has one at a time.  With the
// plan 8 of 512 took 48, now 24, and 32 tokens of 1024 20, now 9.7.
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

constexpr int kThreads = 1024;     // of a workgroup that chooses
constexpr int kPlace = 512, kWaves = kPlace / 64;  // of one that places
constexpr int kMaxE = 1024;
constexpr int kBlockTokens = 64;   // tokens a workgroup chooses for at a time with 16 lanes to each
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

// Keys that order like the numbers: NaN above all, -0 as 0, -inf kNone or
// below (as places past the last expert), which is never chosen.
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 is 0
  const uint32_t key = u ^ (uint32_t)((int)u >> 31 | (int)0x80000000);
  return x != x ? 0xFFFFFFFFu : key;
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

__device__ __forceinline__ float of_key(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __builtin_nanf("");
  return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k);
}

// exp(d) for d <= 0 (or NaN), 0 below the normal range: the product with
// log2(e) in two parts, so that the error stays at a few 2^-24 for any d.  It is
// a term of a sum of at least 1, of which 1024 terms below 2^-126 are no part
// (with expf the weights of 16384 tokens are as far from their 64-bit values,
// 6.9e-8 of their norm, and take 15.6 us against 15.2).
__device__ __forceinline__ float exp_term(float d) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;
  d = d < -200.0f ? -200.0f : d;
  const float t = d * kHi;
  const float rest = __builtin_fmaf(d, kHi, -t) + d * kLo;
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, rest * kLn2, p);
}

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
  int32_t* hist;      // [workgroups][E], rows a multiple of 4 apart
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

constexpr int kCandidates = 64;
// Of the G lanes of a token; an entry is a key and the expert's complement.
struct Candidates {
  uint64_t all[kCandidates], chosen[16];
};

// Lane j % G of a token keeps its choice j in word j / G.
template <int W>
struct Choice {
  uint32_t key[W];
  int expert[W];
};

// The choices by k searches; the largest key (kNone or below: none).
template <int G, int V>
__device__ __forceinline__ uint32_t search(uint32_t (&key)[V], int k, Choice<64 / G>& c) {
  const int l = threadIdx.x % G;
  uint32_t best = 0, top = 0;
  int slot = 0;  // the lane's best, the lower expert among equals
  auto rescan = [&] {
    best = key[0];
    slot = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        slot = i;
      }
  };
  rescan();
#pragma unroll
  for (int w = 0; w < 64 / G; ++w) {
    for (int j = w * G; j < min(k, (w + 1) * G); ++j) {
      const uint32_t most = max_of<G>(best);
      if (most <= kNone) break;  // the same in all G lanes
      const uint32_t e = min_of<G>(best == most ? (uint32_t)(l + slot * G) : 0xFFFFFFFFu);
      if (j == 0) top = most;
      if (l == j - w * G) {
        c.key[w] = most;
        c.expert[w] = (int)e;
      }
      if (best == most && (uint32_t)(l + slot * G) == e) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = i == slot ? 0 : key[i];
        rescan();
      }
    }
  }
  return top;
}

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

template <int CTRL>
__device__ __forceinline__ int shifted(int v) {  // from the lane CTRL - 0x110 before, 0 into a row's first
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// The choices by candidates, k <= 16; false (in every lane of the wave, nothing
// chosen) where a token of the wave has too many.
template <int G, int V>
__device__ __forceinline__ bool select(const uint32_t (&key)[V], int k, Candidates& lds, Choice<64 / G>& c,
                                       uint32_t& top) {
  const int l = threadIdx.x % G;
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = max(best, key[i]);
  if constexpr (G == 64) {  // of the four lanes l, l + 16, ...: every row of 16 has the same
    best = max(best, (uint32_t)__shfl_xor((int)best, 16));
    best = max(best, (uint32_t)__shfl_xor((int)best, 32));
  }
  // how many of the row have a larger one
  int above = 0;
  auto turn = [&](auto n) { above += dpp<0x120 + decltype(n)::value>(best) > best; };
  using std::integral_constant;
  turn(integral_constant<int, 1>{});
  turn(integral_constant<int, 2>{});
  turn(integral_constant<int, 3>{});
  turn(integral_constant<int, 4>{});
  turn(integral_constant<int, 5>{});
  turn(integral_constant<int, 6>{});
  turn(integral_constant<int, 7>{});
  turn(integral_constant<int, 8>{});
  turn(integral_constant<int, 9>{});
  turn(integral_constant<int, 10>{});
  turn(integral_constant<int, 11>{});
  turn(integral_constant<int, 12>{});
  turn(integral_constant<int, 13>{});
  turn(integral_constant<int, 14>{});
  turn(integral_constant<int, 15>{});
  const uint32_t bound = max(min_of<16>(above < k ? best : 0xFFFFFFFFu), kNone + 1);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) mine += key[i] >= bound;
  int end = mine, n;  // inclusive sum over the lanes, and the last one's
  if constexpr (G == 64) {
    end = wave_scan(mine);
    n = __builtin_amdgcn_readlane(end, 63);
  } else {
    end += shifted<0x111>(end);
    end += shifted<0x112>(end);
    end += shifted<0x114>(end);
    end += shifted<0x118>(end);
    n = (int)max_of<16>((uint32_t)end);
  }
  if (__any(n > kCandidates)) return false;
  int at = end - mine;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (key[i] >= bound) lds.all[at++] = (uint64_t)key[i] << 32 | (uint32_t)~(l + i * G);
  wave_sync();
  for (int w = l; w < n; w += G) {
    const uint64_t own = lds.all[w];
    int before = 0;
    // (four at a time, whose reads are in flight together, 6.6 us for 32 tokens
    // against 7.2 one by one or with eight; what lies behind the last candidate
    // is masked)
    for (int i = 0; i < n; i += 4) {
      uint64_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = lds.all[i + q];
#pragma unroll
      for (int q = 0; q < 4; ++q) before += (v[q] > own) & (i + q < n);
    }
    if (before < k) lds.chosen[before] = own;
  }
  wave_sync();
  const int chosen = min(n, k);
  if (l < chosen) {
    c.key[0] = (uint32_t)(lds.chosen[l] >> 32);
    c.expert[0] = (int)~(uint32_t)lds.chosen[l];
  }
  top = chosen > 0 ? (uint32_t)(lds.chosen[0] >> 32) : 0;
  wave_sync();  // written again for the next token
  return true;
}

// Token t by the G lanes that call it; its experts are counted in `count`, and
// left in `local` too where that is given.
template <bool BF16, int G, int V>
__device__ __forceinline__ void choose(const Route& r, int64_t t, int32_t* __restrict__ experts, int* count,
                                       int* local, Candidates& lds) {
  const int l = threadIdx.x % G;
  float x[V];
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = l + i * G < r.E ? load<BF16>(r.logits, t * r.ld + l + i * G) : -__builtin_inff();
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = key_of(x[i]);
  constexpr int W = 64 / G;
  Choice<W> c;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    c.key[w] = 0;
    c.expert[w] = -1;
  }
  uint32_t top = 0;
  bool done = false;
  if (r.k <= 16) done = select<G, V>(key, r.k, lds, c, top);
  if (!done) top = search<G, V>(key, r.k, c);
  const float m = top > kNone ? of_key(top) : 0.0f;
  float sum = 0.0f, p[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    p[w] = c.expert[w] >= 0 ? expf(of_key(c.key[w]) - m) : 0.0f;
    sum += p[w];
  }
  if (!r.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += exp_term(x[i] - m);  // -inf adds 0
  }
  sum = sum_of<G>(sum);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int j = w * G + l;
    if (j < r.k) {
      r.gates[t * r.k + j] = c.expert[w] >= 0 ? p[w] / sum : 0.0f;
      experts[t * r.k + j] = c.expert[w];
      if (local) local[t * r.k + j] = c.expert[w];
      if (c.expert[w] >= 0) atomicAdd(&count[c.expert[w]], 1);
    }
  }
}

// ---- placing ----------------------------------------------------------------

constexpr int kStaged = 4 * kPlace;
struct PlaceLds {
  int slots[kStaged];        // a workgroup's experts, where it has no more
  int count[kWaves][kMaxE];  // rows of an expert in a wave's part, then where the next one goes
  int4 all[kPlace], before[kPlace];
  int scan[kWaves];
};

// Rows of each expert in all workgroups and in those before b, left in
// all[e], before[e] (as arrays of int): columns of four experts to a thread,
// the workgroups' counts dealt to the threads that have the same ones.
__device__ __forceinline__ void add_up(const Sort& s, int b, int nb, PlaceLds& lds) {
  const int columns = (s.E + 3) / 4;
  const int shift = 32 - __builtin_clz(columns) - ((columns & (columns - 1)) == 0);  // columns <= 2^shift
  const int parts = min(kPlace >> shift, 16);
  const int q = threadIdx.x & ((1 << shift) - 1), part = threadIdx.x >> shift;
  int4 all = make_int4(0, 0, 0, 0), before = all;
  if (q < columns && part < parts) {
    const int4* h = reinterpret_cast<const int4*>(s.hist) + q;
#pragma unroll 32
    for (int i = part; i < nb; i += parts) {
      const int4 v = h[(int64_t)i * columns];
      const int in = i < b ? -1 : 0;
      all = make_int4(all.x + v.x, all.y + v.y, all.z + v.z, all.w + v.w);
      before = make_int4(before.x + (v.x & in), before.y + (v.y & in), before.z + (v.z & in), before.w + (v.w & in));
    }
  }
  if (part < parts) {
    lds.all[threadIdx.x] = all;
    lds.before[threadIdx.x] = before;
  }
  __syncthreads();
  int sum[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = threadIdx.x + u * kPlace;
    sum[u][0] = sum[u][1] = 0;
    if (e < s.E) {
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        sum[u][0] += reinterpret_cast<const int*>(lds.all)[(i << (shift + 2)) + e];
        sum[u][1] += reinterpret_cast<const int*>(lds.before)[(i << (shift + 2)) + e];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = threadIdx.x + u * kPlace;
    if (e < s.E) {
      reinterpret_cast<int*>(lds.all)[e] = sum[u][0];
      reinterpret_cast<int*>(lds.before)[e] = sum[u][1];
    }
  }
}

// Workgroup b of nb, the first kPlace threads of it (the others only keep the
// barriers).  slots: the workgroup's experts.
template <bool ALONE>
__device__ __forceinline__ void place(const Sort& s, int b, int nb, const int32_t* slots, PlaceLds& lds) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, E = s.E;
  const bool works = tid < kPlace;
  const int64_t first = (int64_t)b * s.per_block * s.k;
  const int64_t n = min(s.per_block, s.T - b * s.per_block) * s.k;  // slots of this workgroup
  const int64_t part = (n + kPlace - 1) / kPlace * 64;               // and of a wave
  const int64_t lo = works ? min(n, w * part) : n, hi = min(n, lo + part);
  // (asked for first, and there when the counts are added up)
  const bool staged = !ALONE && n <= kStaged;
  int ahead4[kStaged / kPlace];
  if (!ALONE) {
#pragma unroll
    for (int i = 0; i < kStaged / kPlace; ++i) ahead4[i] = staged && tid + i * kPlace < n ? slots[tid + i * kPlace] : -1;
  }
  if (works)
    for (int e = tid; e < E; e += kPlace)
#pragma unroll
      for (int i = 0; i < kWaves; ++i) lds.count[i][e] = 0;
  if (!ALONE) {
    add_up(s, b, nb, lds);
#pragma unroll
    for (int i = 0; i < kStaged / kPlace; ++i) lds.slots[tid + i * kPlace] = ahead4[i];
  }
  auto slot = [&](int64_t i) { return staged ? lds.slots[i] : slots[i]; };
  __syncthreads();
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const int e = slot(i);
    if ((unsigned)e < (unsigned)E) atomicAdd(&lds.count[w][e], 1);
  }
  __syncthreads();
  int64_t base = 0;  // rows of the experts before those of this turn
  for (int e0 = 0; e0 < E; e0 += kPlace) {
    const int e = e0 + tid;
    const bool have = works && e < E;
    int all = 0, before = 0;
    if (have) {
      if (ALONE) {
#pragma unroll
        for (int i = 0; i < kWaves; ++i) all += lds.count[i][e];
      } else {
        all = reinterpret_cast<const int*>(lds.all)[e];
        before = reinterpret_cast<const int*>(lds.before)[e];
      }
    }
    const int sum = wave_scan(all);  // over the wave's experts, inclusive
    if (works && lane == 63) lds.scan[w] = sum;
    __syncthreads();
    int earlier = 0, whole = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      earlier += i < w ? lds.scan[i] : 0;
      whole += lds.scan[i];
    }
    const int64_t start = base + earlier + sum - all;
    if (have) {
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
  for (int64_t r = base + (int64_t)b * blockDim.x + tid; r < R; r += (int64_t)nb * blockDim.x) s.p.row_index[r] = -1;
  const int bits = 32 - __builtin_clz(E);  // E <= 2^bits - 1 tells an empty slot from the experts
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    int e = i < hi ? slot(i) : -1;
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

__device__ __forceinline__ void write_counts(const Sort& s, const int* count, int threads) {
  const int stride = (s.E + 3) / 4 * 4;
  for (int e = threadIdx.x; e < stride; e += threads)
    s.hist[(int64_t)blockIdx.x * stride + e] = e < s.E ? count[e] : 0;
}

// ALONE: one workgroup has all tokens, chooses and places.
template <bool BF16, int G, int V, bool ALONE>
__global__ __launch_bounds__(kThreads) void route_kernel(Route r, Sort s) {
  constexpr int kGroups = kThreads / G;
  __shared__ int count[kMaxE];
  __shared__ int slots[ALONE ? kBlockTokens * 64 : 1];
  for (int e = threadIdx.x; e < r.E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t end = min(r.T, (int64_t)(blockIdx.x + 1) * s.per_block);
  __shared__ Candidates candidates[kGroups];
  for (int64_t t = (int64_t)blockIdx.x * s.per_block + threadIdx.x / G; t < end; t += kGroups)
    choose<BF16, G, V>(r, t, s.p.experts, count, ALONE ? slots : nullptr, candidates[threadIdx.x / G]);
  __syncthreads();
  if constexpr (ALONE) {
    __shared__ PlaceLds lds;
    place<true>(s, 0, 1, slots, lds);
  } else {
    write_counts(s, count, kThreads);
  }
}

__global__ __launch_bounds__(kPlace) void count_kernel(Sort s) {
  __shared__ int count[kMaxE];
  for (int e = threadIdx.x; e < s.E; e += kPlace) count[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * s.per_block, last = min(s.T, first + s.per_block);
  for (int64_t i = first * s.k + threadIdx.x; i < last * s.k; i += kPlace) {
    const int e = s.p.experts[i];
    if ((unsigned)e < (unsigned)s.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  write_counts(s, count, kPlace);
}

template <bool ALONE>
__global__ __launch_bounds__(kPlace) void place_kernel(Sort s) {
  __shared__ PlaceLds lds;
  place<ALONE>(s, blockIdx.x, gridDim.x, s.p.experts + (int64_t)blockIdx.x * s.per_block * s.k, lds);
}

__global__ __launch_bounds__(kPlace) void no_tokens_kernel(int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += kPlace) offsets[e] = 0;
}

// ---- the weights' gradient --------------------------------------------------

template <bool BF16, int G, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ dgates, const void* logits,
                                                             int64_t ld, const float* __restrict__ gates,
                                                             const int32_t* __restrict__ experts, int64_t T, int E,
                                                             int k, int renormalize, void* dlogits, int64_t ld_d) {
  __shared__ float rows[256 / G][G * V];
  const int l = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (t >= T) return;
  float* row = rows[threadIdx.x / G];
  float x[V], p[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = !renormalize && l + i * G < E ? load<BF16>(logits, t * ld + l + i * G) : -__builtin_inff();
    p[i] = 0.0f;
  }
  float dot = 0.0f;
  uint32_t some = 0;
  for (int j = l; j < k; j += G)
    if ((unsigned)experts[t * k + j] < (unsigned)E) {
      dot += gates[t * k + j] * dgates[t * k + j];
      some = 1;
    }
  dot = sum_of<G>(dot);
  // (without an expert the gradient is 0, also where a logit is no number)
  if (!renormalize && max_of<G>(some)) {
    // the maximum is that of the numbers; a NaN or +inf makes the sum NaN as in the forward pass
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, key_of(x[i]));
    top = max_of<G>(top);
    if (top > kNone) {
      const float m = of_key(top);
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
  // the chosen experts' terms through LDS (an expert that is named more than
  // once gets their sum; one wave adds them, whatever else runs)
#pragma unroll
  for (int i = 0; i < V; ++i) row[l + i * G] = p[i];
  wave_sync();
  for (int j = l; j < k; j += G) {
    const int e = experts[t * k + j];
    if ((unsigned)e < (unsigned)E) {
      const float g = gates[t * k + j], dg = dgates[t * k + j];
      unsafeAtomicAdd(&row[e], renormalize ? g * (dg - dot) : g * dg);
    }
  }
  wave_sync();
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (l + i * G < E) store<BF16>(dlogits, t * ld_d + l + i * G, row[l + i * G]);
}

Sort sort_of(int64_t T, int E, int k, const Plan& p, int32_t* ws) {
  const int64_t blocks = std::max<int64_t>(sort_blocks(T), 1);
  return Sort{T, E, k, (T + blocks - 1) / blocks, p, ws};
}

int no_tokens(int32_t* offsets, int E, hipStream_t s) {
  hipLaunchKernelGGL(no_tokens_kernel, dim3(1), dim3(kPlace), 0, s, offsets, E);
  return check_launch();
}

// f(bool_constant<BF16>, G, V) for rows of E logits.  From 65 logits on a token
// has a whole wave; with NARROW only where `whole` says so, or from 257 on.
template <bool NARROW, class F>
int by_width(bool bf16, int E, bool whole, F f) {
  auto with = [&](auto b) {
    using std::integral_constant;
    if (E <= 16) return f(b, integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (E <= 64) return f(b, integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (E <= 256 && whole) return f(b, integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if constexpr (NARROW) {
      if (E <= 128) return f(b, integral_constant<int, 16>{}, integral_constant<int, 8>{});
      if (E <= 256) return f(b, integral_constant<int, 16>{}, integral_constant<int, 16>{});
    }
    if (E <= 512) return f(b, integral_constant<int, 64>{}, integral_constant<int, 8>{});
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
  // As many tokens as a workgroup has waves: a wave each (8 tokens of 256 4.9 us
  // against 6.2 with 16 lanes each, 16 5.5 against 6.3; 32 are even, 64 11.5
  // against 7.7).  Not where the sum is over all E, or over more chosen ones
  // than 16 lanes have, whose order is the lanes': a token's weights would depend
  // on how many others there are.
  const int rc = by_width<true>(logits.bf16, E, renormalize && k <= 16 && T <= kThreads / 64, [&](auto b, auto G, auto V) {
    if (blocks == 1)
      hipLaunchKernelGGL((route_kernel<b.value, G.value, V.value, true>), dim3(1), dim3(kThreads), 0, s, r, sort);
    else
      hipLaunchKernelGGL((route_kernel<b.value, G.value, V.value, false>), dim3(blocks), dim3(kThreads), 0, s, r, sort);
    return check_launch();
  });
  if (rc != FP8B_OK || blocks == 1) return rc;
  hipLaunchKernelGGL(place_kernel<false>, dim3(blocks), dim3(kPlace), 0, s, sort);
  return check_launch();
}

int launch_sort(int64_t T, int E, int k, const Plan& p, int32_t* ws, hipStream_t s) {
  if (T == 0) return no_tokens(p.offsets, E, s);
  const Sort sort = sort_of(T, E, k, p, ws);
  const unsigned blocks = (unsigned)((T + sort.per_block - 1) / sort.per_block);
  if (blocks == 1) {
    hipLaunchKernelGGL(place_kernel<true>, dim3(1), dim3(kPlace), 0, s, sort);
    return check_launch();
  }
  hipLaunchKernelGGL(count_kernel, dim3(blocks), dim3(kPlace), 0, s, sort);
  if (const int rc = check_launch()) return rc;
  hipLaunchKernelGGL(place_kernel<false>, dim3(blocks), dim3(kPlace), 0, s, sort);
  return check_launch();
}

int launch_route_backward(const float* dgates, const Mat& logits, const float* gates, const int32_t* experts, int64_t T,
                          int E, int k, bool renormalize, const Mat& dlogits, hipStream_t s) {
  // (256 tokens of 256 2.6 us against 3.6 with 16 lanes each, 4096 4.3 against 4.9,
  // 16384 9.7 against 9.4)
  return by_width<false>(dlogits.bf16, E, true, [&](auto b, auto G, auto V) {
    const unsigned blocks = (unsigned)((T + 256 / G.value - 1) / (256 / G.value));
    hipLaunchKernelGGL((route_backward_kernel<b.value, G.value, V.value>), dim3(blocks), dim3(256), 0, s, dgates,
                       logits.p, logits.ld, gates, experts, T, E, k, (int)renormalize, dlogits.p, dlogits.ld);
    return check_launch();
  });
}

}  // namespace fp8moe

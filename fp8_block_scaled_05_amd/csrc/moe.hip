// Mixture-of-experts routing for gfx950: the router, its gradient, and the
// dispatch of token rows to the experts as the A operand of the grouped GEMM.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "device.hpp"
#include "fp8bs_decoder.h"
#include "status.hpp"

namespace fp8bs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr float kNegInf = -__builtin_huge_valf();

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  if constexpr (kBf16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[at]) << 16);
  else return static_cast<const float*>(p)[at];
}

// Reductions over the kL = 16 or 64 lanes that hold one token: rotations
// within a row of 16 lanes, then swaps of rows and of halves.
template <int kL, typename T, typename F>
__device__ __forceinline__ T team_reduce(T v, F f) {
  static_assert(sizeof(T) == 4 && (kL == 16 || kL == 64), "");
  auto rot = [&](auto ctrl) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, false);
    v = f(v, __builtin_bit_cast(T, o));
  };
  rot(std::integral_constant<int, 0x128>{});   // row_ror:8
  rot(std::integral_constant<int, 0x124>{});
  rot(std::integral_constant<int, 0x122>{});
  rot(std::integral_constant<int, 0x121>{});
  if constexpr (kL == 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = f(__builtin_bit_cast(T, uint32_t(a[0])), __builtin_bit_cast(T, uint32_t(a[1])));
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    v = f(__builtin_bit_cast(T, uint32_t(b[0])), __builtin_bit_cast(T, uint32_t(b[1])));
  }
  return v;
}
template <int kL> __device__ __forceinline__ float team_max(float v) { return team_reduce<kL>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int kL> __device__ __forceinline__ float team_sum(float v) { return team_reduce<kL>(v, [](float a, float b) { return a + b; }); }
template <int kL> __device__ __forceinline__ uint32_t team_max(uint32_t v) { return team_reduce<kL>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; }); }
template <int kL> __device__ __forceinline__ int team_min(int v) { return team_reduce<kL>(v, [](int a, int b) { return a < b ? a : b; }); }
template <int kL>
__device__ __forceinline__ double team_sum(double v) {
#pragma unroll
  for (int d = kL / 2; d; d >>= 1) v += __shfl_xor(v, d, kL);
  return v;
}

// The kN logits of one lane: runs of kV, one 16-byte load each where rows are
// aligned to it (else kV = 1).
template <int kL, int kN, int kV>
struct Lanes {
  int lane;
  __device__ __forceinline__ int expert(int i) const { return ((i / kV) * kL + lane) * kV + i % kV; }
  template <bool kBf16>
  __device__ __forceinline__ void load(const void* row, int experts, float (&x)[kN]) const {
#pragma unroll
    for (int i = 0; i < kN; i += kV) {
      const int e = expert(i);
      if (e < experts) {
        if constexpr (kV == 1) {
          x[i] = load_logit<kBf16>(row, e);
        } else if constexpr (kBf16) {
          uint32_t u[kV / 2];
          __builtin_memcpy(u, __builtin_assume_aligned(static_cast<const uint16_t*>(row) + e, kV * 2), kV * 2);
#pragma unroll
          for (int j = 0; j < kV / 2; ++j) { x[i + 2 * j] = bf16_lo(u[j]); x[i + 2 * j + 1] = bf16_hi(u[j]); }
        } else {
          __builtin_memcpy(&x[i], __builtin_assume_aligned(static_cast<const float*>(row) + e, kV * 4), kV * 4);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) x[i + j] = kNegInf;
      }
    }
  }
  template <bool kBf16>
  __device__ __forceinline__ void store(void* row, int experts, const float (&x)[kN]) const {
#pragma unroll
    for (int i = 0; i < kN; i += kV) {
      const int e = expert(i);
      if (e >= experts) continue;
      if constexpr (kBf16) {
        __bf16 y[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = static_cast<__bf16>(x[i + j]);
        __builtin_memcpy(__builtin_assume_aligned(static_cast<__bf16*>(row) + e, kV * 2), y, kV * 2);
      } else {
        __builtin_memcpy(__builtin_assume_aligned(static_cast<float*>(row) + e, kV * 4), &x[i], kV * 4);
      }
    }
  }
};

// A float as an integer in the same order; NaN is 1, below every number, and
// 0 stands for what cannot be chosen.
__device__ __forceinline__ uint32_t order_key(float b) {
  const uint32_t u = __float_as_uint(b + 0.0f);          // -0 and +0 tie
  return b != b ? 1u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ double sigmoid64(float x) { return 1.0 / (1.0 + exp(-double(x))); }
__device__ __forceinline__ double below64(float x, float top) { return exp(double(x) - double(top)); }

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t tokens, ld;
  float scale;
  int experts, groups, top_groups, top_k;
  bool renorm;
  int share;            // lanes that look for one group's two best
  int size;             // experts of a group
  uint32_t per_size;    // 2^21 / size, rounded up: e / size = e per_size >> 21 for e, size <= 1024
  __device__ __forceinline__ int group_of(int e) const { return __umul24(e, per_size) >> 21; }
};

// kL lanes a token, kN experts a lane.  The choice is made by top_k rounds of
// a maximum over the ordered scores and a minimum over the indexes that hold
// it; the weights are then evaluated again at the chosen experts only.  Bound
// by vector instructions: the 64-bit exponential and quotient of every expert
// and the rounds (32768 tokens of 256 experts 30 us, 1.2 TB/s).
template <int kL, int kN, int kV, bool kBf16, bool kSoftmax>
__global__ __launch_bounds__(256) void route_kernel(RouteParams p) {
  constexpr int kTeams = 256 / kL;
  constexpr int kSlots = kL == 16 ? 2 : 1;               // choices that a lane holds
  __shared__ float sh_b[kTeams][kL * kN + 64];
  __shared__ uint32_t sh_mark[kTeams][64];
  const int team = threadIdx.x / kL;
  const Lanes<kL, kN, kV> at{static_cast<int>(threadIdx.x % kL)};
  const int lane = at.lane, experts = p.experts;
  const int64_t t_raw = int64_t(blockIdx.x) * kTeams + team;
  const int64_t t = min(t_raw, p.tokens - 1);            // a team past the end repeats the last token and writes nothing
  const char* row = static_cast<const char*>(p.logits) + t * p.ld * (kBf16 ? 2 : 4);
  float x[kN];
  at.template load<kBf16>(row, experts, x);
  float top = 0.0f;
  double sum = 0.0;              // softmax: its inverse, after the sum
  float b[kN];
  if constexpr (kSoftmax) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) top = fmaxf(top, x[i]);
    top = team_max<kL>(top);
    double w[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      w[i] = at.expert(i) < experts ? below64(x[i], top) : 0.0;
      sum += w[i];
    }
    sum = 1.0 / team_sum<kL>(sum);
#pragma unroll
    for (int i = 0; i < kN; ++i) b[i] = static_cast<float>(w[i] * sum);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) b[i] = static_cast<float>(sigmoid64(x[i]));
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < kN; i += kV) {
      const float* from = p.bias + min(at.expert(i), experts - kV);    // what experts past the end get is not looked at
      float add[kV];
      __builtin_memcpy(add, __builtin_assume_aligned(from, 4 * kV), 4 * kV);
#pragma unroll
      for (int j = 0; j < kV; ++j) b[i + j] += add[j];
    }
  }
  uint64_t kept = ~uint64_t(0);
  if (p.groups > 1) {
    const int size = p.size;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = at.expert(i);
      sh_b[team][e + min(p.group_of(e), 63)] = b[i];       // groups start at different banks
    }
    __builtin_amdgcn_wave_barrier();
    // `share` lanes a group, each over every share-th expert of it
    const int g = lane / p.share, part = lane - g * p.share;
    float m1 = kNegInf, m2 = kNegInf;
    if (g < p.groups) {
#pragma unroll 4
      for (int i = part; i < size; i += p.share) {
        const float v = fmaxf(sh_b[team][g * (size + 1) + i], kNegInf);     // a NaN counts as -infinity
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    }
    for (int d = 1; d < p.share; d <<= 1) {
      const float o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
      m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
      m1 = fmaxf(m1, o1);
    }
    const uint32_t mark = g < p.groups ? order_key(size > 1 ? m1 + m2 : m1) : 0u;
    if (part == 0 && g < p.groups) sh_mark[team][g] = mark;
    __builtin_amdgcn_wave_barrier();
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const uint32_t other = sh_mark[team][o];
      rank += other > mark || (other == mark && o < g);
    }
    uint64_t mine = part == 0 && g < p.groups && rank < p.top_groups ? uint64_t(1) << g : 0;
    uint32_t lo = static_cast<uint32_t>(mine), hi = static_cast<uint32_t>(mine >> 32);
    lo = team_reduce<kL>(lo, [](uint32_t a, uint32_t c) { return a | c; });
    if (kL == 64 && p.groups > 32) hi = team_reduce<kL>(hi, [](uint32_t a, uint32_t c) { return a | c; });
    kept = uint64_t(hi) << 32 | lo;
  }
  uint32_t key[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = at.expert(i);
    const int g = p.groups > 1 ? p.group_of(e) : 0;
    const bool in = e < experts && ((kL == 16 ? static_cast<uint32_t>(kept) >> (g & 31) : static_cast<uint32_t>(kept >> (g & 63))) & 1);
    key[i] = in ? order_key(b[i]) : 0u;
  }
  int my_id[kSlots] = {};           // lane j holds choices j and j + kL
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) best = key[i] > best ? key[i] : best;
    best = team_max<kL>(best);
    int e = 0x7fffffff;
#pragma unroll
    for (int i = kN - 1; i >= 0; --i) e = key[i] == best ? at.expert(i) : e;
    e = team_min<kL>(e);
#pragma unroll
    for (int i = 0; i < kN; ++i) key[i] = e == at.expert(i) ? 0u : key[i];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) my_id[s] = j == lane + s * kL ? e : my_id[s];
  }
  float w[kSlots], total = 0.0f;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    w[s] = 0.0f;
    if (lane + s * kL < p.top_k) {
      const float y = load_logit<kBf16>(row, my_id[s]);
      w[s] = static_cast<float>(kSoftmax ? below64(y, top) * sum : sigmoid64(y));
    }
    total += w[s];
  }
  if (p.renorm) total = team_sum<kL>(total) + 1e-20f;
  if (t_raw >= p.tokens) return;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kL;
    if (j < p.top_k) {
      p.ids[t * p.top_k + j] = my_id[s];
      p.weights[t * p.top_k + j] = (p.renorm ? w[s] / total : w[s]) * p.scale;
    }
  }
}

struct RouteGradParams {
  const float* grad;
  const void* logits;
  const int32_t* ids;
  void* dlogits;
  int64_t tokens, ld, ld_d;
  float scale;
  int experts, top_k;
  bool renorm;
};

// kL lanes a token, kN experts a lane.  Softmax is bound by the exponentials of
// all kN (32768 tokens, bf16: 160 experts 10.0 us, 4.4 by their bytes, 256
// experts 11.2 and 7.2).  Sigmoid reads the chosen logits alone and writes rows
// that are mostly 0 (256 experts, float32 10.2 us, 7.2 by the bytes; bf16 8.0
// and 3.9).
template <int kL, int kN, int kV, bool kBf16, bool kSoftmax>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradParams p) {
  constexpr int kTeams = 256 / kL;
  constexpr int kSlots = kL == 16 ? 2 : 1;
  __shared__ __align__(16) float sh_add[kTeams][kL * kN];
  const Lanes<kL, kN, kV> at{static_cast<int>(threadIdx.x % kL)};
  const int lane = at.lane, experts = p.experts;
  const int64_t t_raw = int64_t(blockIdx.x) * kTeams + threadIdx.x / kL;
  const int64_t t = min(t_raw, p.tokens - 1);
  const char* row = static_cast<const char*>(p.logits) + t * p.ld * (kBf16 ? 2 : 4);
  // lane j holds choices j and j + kL
  int id[kSlots];
  float g[kSlots], w[kSlots], rest[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kL;
    id[s] = -1;
    g[s] = w[s] = rest[s] = 0.0f;
    if (j < p.top_k) {
      id[s] = p.ids[t * p.top_k + j];
      g[s] = p.grad[t * p.top_k + j] * p.scale;
    }
    if (id[s] < 0 || id[s] >= experts) {
      id[s] = -1;
      g[s] = 0.0f;
    }
  }
  float d[kN], top = 0.0f, sum = 1.0f;
  if constexpr (kSoftmax) {
    at.template load<kBf16>(row, experts, d);
    top = d[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) top = fmaxf(top, d[i]);
    top = team_max<kL>(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      d[i] = expf(d[i] - top);
      sum += d[i];
    }
    sum = team_sum<kL>(sum);
  }
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (id[s] < 0) continue;
    const float x = load_logit<kBf16>(row, id[s]);
    if constexpr (kSoftmax) {
      w[s] = expf(x - top) / sum;
    } else {
      w[s] = 1.0f / (1.0f + expf(-x));
      rest[s] = 1.0f / (1.0f + expf(x));
    }
  }
  if (p.renorm) {
    float total = 0.0f, mean = 0.0f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) total += w[s];
    total = team_sum<kL>(total) + 1e-20f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) mean += g[s] * (w[s] / total);
    mean = team_sum<kL>(mean);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) g[s] = id[s] >= 0 ? (g[s] - mean) / total : 0.0f;
  }
  float add[kSlots], dot = 0.0f;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    add[s] = g[s] * w[s];
    dot += add[s];
    if (!kSoftmax) add[s] *= rest[s];
  }
  if constexpr (kSoftmax) {
    const float f = -team_sum<kL>(dot) / sum;
#pragma unroll
    for (int i = 0; i < kN; ++i) d[i] *= f;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) d[i] = 0.0f;
  }
  // to their experts through LDS: a choice that stands before others of the
  // same expert brings all their sums, in the order of the choices
  float* mine = sh_add[threadIdx.x / kL];
#pragma unroll
  for (int i = 0; i < kN; ++i) mine[at.expert(i)] = 0.0f;
  float all[kSlots] = {};
  bool first[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) first[s] = id[s] >= 0;
#pragma unroll
  for (int so = 0; so < kSlots; ++so) {
    for (int j = 0; j < kL && j + so * kL < p.top_k; ++j) {
      const int e = __shfl(id[so], j, kL);
      const float a = __shfl(add[so], j, kL);
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        if (e != id[s]) continue;
        all[s] += a;
        if (j + so * kL < lane + s * kL) first[s] = false;
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int s = 0; s < kSlots; ++s)
    if (first[s]) mine[id[s]] = all[s];
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < kN; ++i) d[i] += mine[at.expert(i)];
  if (t_raw < p.tokens) at.template store<kBf16>(static_cast<char*>(p.dlogits) + t * p.ld_d * (kBf16 ? 2 : 4), experts, d);
}

// ---------------------------------------------------------------------------
// Dispatch: a stable counting sort of the choices by expert, then the rows.
//
// Few choices (a decode step): one launch.  Each token's workgroup finds the
// places of its choices by counting the choices that come before them.
// Many: the choices fall into chunks of one or more runs of kRun.  A first
// kernel counts each chunk's experts into counts[chunk][expert]; a second one
// adds up the chunks before its own and the experts before each expert, ranks
// its own choices run by run and writes order, position and offsets; a third
// quantizes each token's row once and writes it at its top_k places.  Every
// workgroup of the second reads all counts, so there are at most kMaxChunks
// chunks, one a CU: beyond that their runs grow in number (10^6 tokens of 128
// columns, 8 choices each, 912 us; with chunks of one run 2191).
constexpr int kFew = 4096;
constexpr int kRun = 2048;
constexpr int kMaxChunks = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRunsOf64 = kRun / kSortThreads;

// How n choices (more than kFew) are cut up.
struct Chunks {
  int chunks, runs;      // runs of kRun choices a chunk
  explicit Chunks(int64_t n) {
    const int64_t all = (n + kRun - 1) / kRun;
    runs = static_cast<int>((all + kMaxChunks - 1) / kMaxChunks);
    chunks = static_cast<int>((all + runs - 1) / runs);
  }
};

__device__ __forceinline__ int choice_bin(const int32_t* ids, int64_t i, int experts) {
  const int32_t e = ids[i];
  return e >= 0 && e < experts ? e : experts;
}

// Exclusive sum over a workgroup's threads; `total` is the sum of all.
template <int kThreads>
__device__ __forceinline__ int block_exclusive(int v, int& total) {
  __shared__ int32_t sums[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int up = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  return before + up - v;
}

__global__ __launch_bounds__(kSortThreads) void dispatch_count_kernel(const int32_t* __restrict__ ids, int64_t n, int experts, int runs,
                                                                      int32_t* __restrict__ counts) {
  __shared__ int32_t bins[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= experts; e += kSortThreads) bins[e] = 0;
  __syncthreads();
  const int64_t base = int64_t(blockIdx.x) * runs * kRun;
  for (int run = 0; run < runs; ++run) {
#pragma unroll
    for (int r = 0; r < kRunsOf64; ++r) {
      const int64_t i = base + int64_t(run) * kRun + r * kSortThreads + threadIdx.x;
      if (i < n) atomicAdd(&bins[choice_bin(ids, i, experts)], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += kSortThreads) counts[int64_t(blockIdx.x) * (experts + 1) + e] = bins[e];
}

__global__ __launch_bounds__(kSortThreads) void dispatch_rank_kernel(const int32_t* __restrict__ ids, int64_t n, int experts, int chunks, int runs,
                                                                     const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                                     int32_t* __restrict__ order, int32_t* __restrict__ position) {
  __shared__ int32_t start[kMaxExperts + 1];
  __shared__ uint16_t seen[kSortWaves][kMaxExperts + 2];      // of each wave's choices, then of the waves before it
  const int chunk = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // choices of each expert in earlier chunks and in all
  int total = 0, sum;
  for (int e = tid; e <= experts; e += kSortThreads) {
    int before = 0, all = 0;
#pragma unroll 8
    for (int k = 0; k < chunks; ++k) {
      const int v = counts[int64_t(k) * (experts + 1) + e];
      before += k < chunk ? v : 0;
      all += v;
    }
    start[e] = before;
    if (e < experts) total = all;
  }
  const int first = block_exclusive<kSortThreads>(total, sum);      // expert tid's first place
  __syncthreads();
  if (tid < experts) start[tid] += first;
  if (tid == 0) start[experts] += sum;
  if (chunk == 0) {
    if (tid < experts) offsets[tid] = first;
    if (tid == 0) offsets[experts] = sum;
  }
  for (int run = 0; run < runs; ++run) {
    for (int e = lane; e <= experts; e += 64) seen[wave][e] = 0;
    __builtin_amdgcn_wave_barrier();
    // rank of a choice among its wave's choices of the same expert; a wave
    // takes kRunsOf64 times 64 consecutive choices
    int bin[kRunsOf64], rank[kRunsOf64];
    const int64_t base = (int64_t(chunk) * runs + run) * kRun + wave * (64 * kRunsOf64) + lane;
#pragma unroll
    for (int r = 0; r < kRunsOf64; ++r) bin[r] = base + 64 * r < n ? choice_bin(ids, base + 64 * r, experts) : -1;
#pragma unroll
    for (int r = 0; r < kRunsOf64; ++r) {
      uint64_t same = __ballot(bin[r] >= 0);
#pragma unroll
      for (int bit = 0; bit < 11; ++bit) {
        const bool on = bin[r] >> bit & 1;
        const uint64_t who = __ballot(on);
        same &= on ? who : ~who;
      }
      if (bin[r] >= 0) {
        const int older = seen[wave][bin[r]], lower = __popcll(same & ((uint64_t(1) << lane) - 1));
        rank[r] = older + lower;
        if (lower == 0) seen[wave][bin[r]] = static_cast<uint16_t>(older + __popcll(same));
      }
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    int here[2] = {};                    // the run's choices of expert tid, and of expert kSortThreads
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = tid + i * kSortThreads;
      if (e > experts) break;
      int before = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = seen[w][e];
        seen[w][e] = static_cast<uint16_t>(before);
        before += v;
      }
      here[i] = before;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRunsOf64; ++r) {
      if (bin[r] < 0) continue;
      const int place = start[bin[r]] + seen[wave][bin[r]] + rank[r];
      position[base + 64 * r] = place;
      order[place] = static_cast<int32_t>(base + 64 * r);
    }
    if (run + 1 == runs) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (tid + i * kSortThreads <= experts) start[tid + i * kSortThreads] += here[i];
  }
}

// Eight columns of a row, 16 lanes a tile: codes and the tile's scale.
template <bool kBf16>
__device__ __forceinline__ u32x2 quantize8(const void* __restrict__ x, int64_t at, float& s) {
  float v[8];
  if constexpr (kBf16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at);
    const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  s = tile_scale(row16_max(amax));
  return u32x2{pack4_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s), pack4_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s)};
}
__device__ __forceinline__ void put_tile(uint8_t* q, float* scale, int64_t place, int64_t cols, int64_t col, bool live, u32x2 codes, float s) {
  u32x2* to = reinterpret_cast<u32x2*>(q + place * cols + col);
  __builtin_nontemporal_store(live ? codes : u32x2{0, 0}, to);
  if ((threadIdx.x & 15) == 0) scale[place * (cols / 128) + col / 128] = live ? s : 1.0f;
}

// Workgroup (2048 columns, token).
template <bool kBf16>
__global__ __launch_bounds__(256) void dispatch_rows_kernel(const void* __restrict__ x, int64_t cols, int64_t ld_x, int top_k, int experts,
                                                            const int32_t* __restrict__ ids, const int32_t* __restrict__ position,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int64_t t = blockIdx.y;
  const int64_t col = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (col >= cols) return;
  float s;
  const u32x2 codes = quantize8<kBf16>(x, t * ld_x + col, s);
#pragma unroll 4
  for (int j = 0; j < top_k; ++j)
    put_tile(q, scale, position[t * top_k + j], cols, col, choice_bin(ids, t * top_k + j, experts) < experts, codes, s);
}

// All of a call with at most kFew choices: workgroup (2048 columns, token);
// one more for the offsets.
template <bool kBf16>
__global__ __launch_bounds__(256) void dispatch_few_kernel(const void* __restrict__ x, int64_t cols, int64_t ld_x, int tokens, int top_k,
                                                           int experts, const int32_t* __restrict__ ids, uint8_t* __restrict__ q,
                                                           float* __restrict__ scale, int32_t* __restrict__ offsets,
                                                           int32_t* __restrict__ order, int32_t* __restrict__ position) {
  constexpr int kMine = kFew / 256;
  const int n = tokens * top_k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (static_cast<int>(blockIdx.y) == tokens) {
    if (blockIdx.x) return;
    __shared__ int32_t bins[kMaxExperts + 1];
    constexpr int kEach = (kMaxExperts + 255) / 256;
    for (int e = tid; e <= experts; e += 256) bins[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 256) atomicAdd(&bins[choice_bin(ids, i, experts)], 1);
    __syncthreads();
    int mine = 0, total;
    for (int e = tid * kEach; e < min(experts, (tid + 1) * kEach); ++e) mine += bins[e];
    int at = block_exclusive<256>(mine, total);
    for (int e = tid * kEach; e < min(experts, (tid + 1) * kEach); ++e) {
      offsets[e] = at;
      at += bins[e];
    }
    if (tid == 0) offsets[experts] = total;
    return;
  }
  __shared__ int32_t before[4][kMaxTopK];
  const int t = blockIdx.y;
  const int64_t col = (int64_t(blockIdx.x) * 256 + tid) * 8;
  float s = 1.0f;
  u32x2 codes = {0, 0};
  if (col < cols) codes = quantize8<kBf16>(x, t * ld_x + col, s);
  int bin[kMine];
#pragma unroll
  for (int r = 0; r < kMine; ++r) bin[r] = r * 256 + tid < n ? choice_bin(ids, r * 256 + tid, experts) : 0x7fffffff;
  for (int j = 0; j < top_k; ++j) {
    const int i = t * top_k + j, e = choice_bin(ids, i, experts);
    int count = 0;
#pragma unroll
    for (int r = 0; r < kMine; ++r) {
      if (r * 256 >= n) break;
      count += __popcll(__ballot(bin[r] < e || (bin[r] == e && r * 256 + tid < i)));
    }
    if (lane == 0) before[wave][j] = count;
  }
  __syncthreads();
#pragma unroll 4
  for (int j = 0; j < top_k; ++j) {
    const int place = (before[0][j] + before[1][j]) + (before[2][j] + before[3][j]);
    if (col < cols) put_tile(q, scale, place, cols, col, choice_bin(ids, t * top_k + j, experts) < experts, codes, s);
    if (blockIdx.x == 0 && tid == j) {
      position[t * top_k + j] = place;
      order[place] = t * top_k + j;
    }
  }
}

fp8bs_status check_router(const char* fn, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld, int32_t top_k, int32_t score,
                          double scale) {
  if (!valid_dtype(dtype)) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (score != FP8BS_SCORE_SIGMOID && score != FP8BS_SCORE_SOFTMAX) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown score %d", fn, score);
  if (tokens < 0 || tokens >= (int64_t(1) << 26)) return fail(FP8BS_ERR_INVALID_ARG, "%s: %lld tokens, not 0 to 2^26", fn, (long long)tokens);
  if (experts < 1 || experts > kMaxExperts)
    return fail(FP8BS_ERR_SHAPE, "%s: %lld experts, 1 to %d are supported", fn, (long long)experts, kMaxExperts);
  if (top_k < 1 || top_k > kMaxTopK) return fail(FP8BS_ERR_SHAPE, "%s: top_k %d is not in 1 .. %d", fn, top_k, kMaxTopK);
  if (ld < experts) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch smaller than the row", fn);
  if (!sane_matrix(tokens, ld, elem_size(dtype))) return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes and pitches exceed any allocation", fn);
  if (!std::isfinite(scale)) return fail(FP8BS_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  return FP8BS_OK;
}
// rows of whole, aligned runs of four elements
bool four_wide(const void* p, int32_t dtype, int64_t cols, int64_t ld) {
  return cols % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * elem_size(dtype)) == 0;
}
bool aligned_elem(const void* p, int32_t dtype) { return reinterpret_cast<uintptr_t>(p) % elem_size(dtype) == 0; }

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

// 16 lanes a token where there are enough tokens to fill the chip so: their
// reductions stay within a row of lanes and serve four tokens at once.  With
// few tokens 64 lanes have the shorter path.  256 experts in 8 groups: 32768
// tokens 30.8 us with 16 lanes, 46.0 us with 64; 4096 tokens 8.4 and 8.7; 2048
// tokens 8.1 and 5.9.  384 experts, softmax, 32768 tokens: 36.5 and 51.8 us.
// Up to 384 experts: the gradient takes the same widths, and with 32 experts
// a lane gains nothing more from 16 lanes (512 experts, softmax, 32768 tokens:
// gradient 24.0 us, with 64 lanes 23.0; router 44.1 and 51.9).
constexpr int64_t kNarrowTokens = 4096;
static bool narrow_teams(int64_t tokens, int64_t experts, int groups) {
  return experts <= 384 && groups <= 16 && tokens >= kNarrowTokens;
}
#define FP8BS_KINDS(KERNEL, L, N, V) \
  do { \
    if (bf16) { if (softmax) FP8BS_L((KERNEL<L, N, V, true, true>), L); else FP8BS_L((KERNEL<L, N, V, true, false>), L); } \
    else { if (softmax) FP8BS_L((KERNEL<L, N, V, false, true>), L); else FP8BS_L((KERNEL<L, N, V, false, false>), L); } \
  } while (0)
#define FP8BS_TEAMS(KERNEL, V) \
  do { \
    if (narrow) { \
      if (experts <= 64) FP8BS_KINDS(KERNEL, 16, 4, V); \
      else if (experts <= 128) FP8BS_KINDS(KERNEL, 16, 8, V); \
      else if (experts <= 256) FP8BS_KINDS(KERNEL, 16, 16, V); \
      else FP8BS_KINDS(KERNEL, 16, 24, V); \
    } else { \
      if (experts <= 256) FP8BS_KINDS(KERNEL, 64, 4, V); \
      else if (experts <= 512) FP8BS_KINDS(KERNEL, 64, 8, V); \
      else FP8BS_KINDS(KERNEL, 64, 16, V); \
    } \
  } while (0)

extern "C" fp8bs_status fp8_moe_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld, int32_t score,
                                      const float* bias, int32_t groups, int32_t top_groups, int32_t top_k, int32_t renormalize,
                                      double scale, int32_t* ids, float* weights, hipStream_t stream) {
  const char* fn = "fp8_moe_route";
  if (fp8bs_status st = check_router(fn, dtype, tokens, experts, ld, top_k, score, scale)) return st;
  if (groups < 1 || groups > 64 || experts % groups)
    return fail(FP8BS_ERR_SHAPE, "%s: %lld experts do not fall into %d groups (at most 64)", fn, (long long)experts, groups);
  if (top_groups < 1 || top_groups > groups) return fail(FP8BS_ERR_SHAPE, "%s: top_groups %d is not in 1 .. %d", fn, top_groups, groups);
  if (top_k > top_groups * (experts / groups))
    return fail(FP8BS_ERR_SHAPE, "%s: top_k %d of %lld experts in the groups that stay", fn, top_k, (long long)(top_groups * (experts / groups)));
  if (tokens == 0) return FP8BS_OK;
  if (!logits || !ids || !weights) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned_elem(logits, dtype) || !aligned4(bias) || !aligned4(ids) || !aligned4(weights))
    return fail(FP8BS_ERR_ALIGNMENT, "%s: arrays must be aligned to their elements", fn);
  const bool bf16 = dtype == FP8BS_BF16, softmax = score == FP8BS_SCORE_SOFTMAX, narrow = narrow_teams(tokens, experts, groups);
  const int64_t size = experts / groups;
  int share = 1;
  while (2 * share * groups <= (narrow ? 16 : 64)) share *= 2;
  const RouteParams p{logits, bias, ids, weights, tokens, ld, static_cast<float>(scale), static_cast<int>(experts), groups, top_groups, top_k,
                      renormalize != 0, share, static_cast<int>(size), static_cast<uint32_t>((1 << 21) / size + 1)};
  begin_launch();
#define FP8BS_L(K, L) hipLaunchKernelGGL(K, dim3(static_cast<uint32_t>((tokens + 256 / L - 1) / (256 / L))), dim3(256), 0, stream, p)
  if (four_wide(logits, dtype, experts, ld) && aligned16(bias)) FP8BS_TEAMS(route_kernel, 4);
  else FP8BS_TEAMS(route_kernel, 1);
#undef FP8BS_L
  return check_launch(fn);
}

extern "C" fp8bs_status fp8_moe_route_backward(const float* grad, const void* logits, int32_t dtype, int64_t tokens, int64_t experts,
                                               int64_t ld, const int32_t* ids, int32_t top_k, int32_t score, int32_t renormalize,
                                               double scale, void* dlogits, int64_t ld_d, hipStream_t stream) {
  const char* fn = "fp8_moe_route_backward";
  if (fp8bs_status st = check_router(fn, dtype, tokens, experts, ld, top_k, score, scale)) return st;
  if (ld_d < experts) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch smaller than the row", fn);
  if (!sane_matrix(tokens, ld_d, elem_size(dtype))) return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes and pitches exceed any allocation", fn);
  if (tokens == 0) return FP8BS_OK;
  if (!grad || !logits || !ids || !dlogits) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned_elem(logits, dtype) || !aligned_elem(dlogits, dtype) || !aligned4(grad) || !aligned4(ids))
    return fail(FP8BS_ERR_ALIGNMENT, "%s: arrays must be aligned to their elements", fn);
  const bool bf16 = dtype == FP8BS_BF16, softmax = score == FP8BS_SCORE_SOFTMAX, narrow = narrow_teams(tokens, experts, 1);
  const RouteGradParams p{grad, logits, ids, dlogits, tokens, ld, ld_d, static_cast<float>(scale), static_cast<int>(experts), top_k,
                          renormalize != 0};
  begin_launch();
#define FP8BS_L(K, L) hipLaunchKernelGGL(K, dim3(static_cast<uint32_t>((tokens + 256 / L - 1) / (256 / L))), dim3(256), 0, stream, p)
  if (four_wide(logits, dtype, experts, ld) && four_wide(dlogits, dtype, experts, ld_d)) FP8BS_TEAMS(route_backward_kernel, 4);
  else FP8BS_TEAMS(route_backward_kernel, 1);
#undef FP8BS_L
  return check_launch(fn);
}

extern "C" int64_t fp8_moe_dispatch_workspace(int64_t tokens, int32_t experts, int32_t top_k) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || tokens >= (int64_t(1) << 31) / top_k) {
    fail(FP8BS_ERR_SHAPE, "fp8_moe_dispatch_workspace: sizes out of range");
    return -1;
  }
  if (tokens * top_k <= kFew) return 0;
  return int64_t(Chunks(tokens * top_k).chunks) * (experts + 1) * 4;
}

extern "C" fp8bs_status fp8_moe_dispatch(const void* x, int32_t x_dtype, int64_t tokens, int64_t cols, int64_t ld_x, const int32_t* ids,
                                         int32_t top_k, int32_t experts, uint8_t* q, float* scale, int32_t* offsets, int32_t* order,
                                         int32_t* position, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const char* fn = "fp8_moe_dispatch";
  if (!valid_dtype(x_dtype)) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown x_dtype %d", fn, x_dtype);
  if (tokens < 0 || cols < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols < 128 || cols % 128) return fail(FP8BS_ERR_SHAPE, "%s: cols %lld not a positive multiple of 128", fn, (long long)cols);
  if (experts < 1 || experts > kMaxExperts) return fail(FP8BS_ERR_SHAPE, "%s: %d experts, 1 to %d are supported", fn, experts, kMaxExperts);
  if (top_k < 1 || top_k > kMaxTopK) return fail(FP8BS_ERR_SHAPE, "%s: top_k %d is not in 1 .. %d", fn, top_k, kMaxTopK);
  if (tokens >= (int64_t(1) << 31) / top_k) return fail(FP8BS_ERR_INVALID_ARG, "%s: 2^31 choices or more", fn);
  if (!offsets) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (offsets)", fn);
  if (tokens > 0 && (!x || !ids || !q || !scale || !order || !position)) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (ld_x < cols) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch smaller than the row", fn);
  const int64_t n = tokens * top_k;
  if (!sane_matrix(tokens, ld_x, elem_size(x_dtype)) || !sane_matrix(n, cols, 1))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes and pitches exceed any allocation", fn);
  if (!aligned16(x) || !aligned16(q) || (ld_x * elem_size(x_dtype)) % 16)
    return fail(FP8BS_ERR_ALIGNMENT, "%s: x, its pitch and q must be 16-byte aligned", fn);
  if (!aligned4(ids) || !aligned4(scale) || !aligned4(offsets) || !aligned4(order) || !aligned4(position))
    return fail(FP8BS_ERR_ALIGNMENT, "%s: scale and index arrays must be 4-byte aligned", fn);
  const int64_t need = fp8_moe_dispatch_workspace(tokens, experts, top_k);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace of %lld bytes is needed, %lld given", fn, (long long)need,
                (long long)(workspace ? workspace_bytes : 0));
  if (!aligned4(workspace)) return fail(FP8BS_ERR_ALIGNMENT, "%s: workspace must be 4-byte aligned", fn);
  begin_launch();
  const uint32_t col_blocks = static_cast<uint32_t>((cols + 2047) / 2048);
  if (n <= kFew) {
    const dim3 grid(col_blocks, static_cast<uint32_t>(tokens + 1));
    if (x_dtype == FP8BS_BF16)
      hipLaunchKernelGGL(dispatch_few_kernel<true>, grid, dim3(256), 0, stream, x, cols, ld_x, static_cast<int>(tokens), top_k, experts, ids, q,
                         scale, offsets, order, position);
    else
      hipLaunchKernelGGL(dispatch_few_kernel<false>, grid, dim3(256), 0, stream, x, cols, ld_x, static_cast<int>(tokens), top_k, experts, ids, q,
                         scale, offsets, order, position);
  } else {
    const Chunks cut(n);
    int32_t* counts = static_cast<int32_t*>(workspace);
    hipLaunchKernelGGL(dispatch_count_kernel, dim3(cut.chunks), dim3(kSortThreads), 0, stream, ids, n, experts, cut.runs, counts);
    hipLaunchKernelGGL(dispatch_rank_kernel, dim3(cut.chunks), dim3(kSortThreads), 0, stream, ids, n, experts, cut.chunks, cut.runs, counts, offsets,
                       order, position);
    for (int64_t t0 = 0; t0 < tokens; t0 += 65535) {
      const int64_t m = std::min<int64_t>(tokens - t0, 65535);
      const dim3 grid(col_blocks, static_cast<uint32_t>(m));
      const char* src = static_cast<const char*>(x) + t0 * ld_x * elem_size(x_dtype);
      if (x_dtype == FP8BS_BF16)
        hipLaunchKernelGGL(dispatch_rows_kernel<true>, grid, dim3(256), 0, stream, src, cols, ld_x, top_k, experts, ids + t0 * top_k,
                           position + t0 * top_k, q, scale);
      else
        hipLaunchKernelGGL(dispatch_rows_kernel<false>, grid, dim3(256), 0, stream, src, cols, ld_x, top_k, experts, ids + t0 * top_k,
                           position + t0 * top_k, q, scale);
    }
  }
  return check_launch(fn);
}

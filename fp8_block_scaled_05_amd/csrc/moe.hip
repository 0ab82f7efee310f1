// Mixture-of-experts routing for gfx950: the router, its gradient, and the
// dispatch of token rows to the experts as the A operand of the grouped GEMM.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

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

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A float's place in descending order with ties to the lower index, as one
// integer to take the maximum of; NaN lies below every number.
__device__ __forceinline__ uint64_t order_key(float b, uint32_t index) {
  uint32_t u = __float_as_uint(b + 0.0f);          // -0 and +0 tie
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  if (b != b) u = 0;
  return (uint64_t(u) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = __shfl_xor(static_cast<unsigned long long>(v), d);
    v = o > v ? o : v;
  }
  return v;
}

// One wave a token; expert e = lane + 64 i.
constexpr int kRouteWaves = 4;
template <int kN, bool kBf16, bool kSoftmax>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(const void* __restrict__ logits, int64_t tokens, int experts, int64_t ld,
                                                                 const float* __restrict__ bias, int groups, int top_groups, int top_k,
                                                                 bool renorm, float scale, int32_t* __restrict__ ids,
                                                                 float* __restrict__ weights) {
  __shared__ float sh_b[kRouteWaves][kN * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = int64_t(blockIdx.x) * kRouteWaves + wave;
  if (t >= tokens) return;
  float score[kN], b[kN];
  double x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < experts ? double(load_logit<kBf16>(logits, t * ld + e)) : -__builtin_huge_val();
  }
  if constexpr (kSoftmax) {
    double top = x[0], sum = 0.0;
#pragma unroll
    for (int i = 1; i < kN; ++i) top = fmax(top, x[i]);
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmax(top, __shfl_xor(top, d));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      x[i] = exp(x[i] - top);
      sum += x[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kN; ++i) score[i] = static_cast<float>(x[i] / sum);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) score[i] = static_cast<float>(1.0 / (1.0 + exp(-x[i])));
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = lane + 64 * i;
    b[i] = e < experts && bias ? score[i] + bias[e] : score[i];
    sh_b[wave][e] = b[i];
  }
  __builtin_amdgcn_wave_barrier();
  uint64_t kept = ~uint64_t(0);
  if (groups > 1) {
    const int size = experts / groups;
    uint64_t mark = 0;
    if (lane < groups) {
      float m1 = kNegInf, m2 = kNegInf;
      for (int i = 0; i < size; ++i) {
        const float v = sh_b[wave][lane * size + i];
        if (v > m1) { m2 = m1; m1 = v; }
        else if (v > m2) m2 = v;
      }
      mark = order_key(size > 1 ? m1 + m2 : m1, lane);
    }
    kept = 0;
    for (int i = 0; i < top_groups; ++i) {
      const uint64_t best = wave_max_u64(mark);
      if (mark == best) mark = 0;
      kept |= uint64_t(1) << (0xffffffffu - uint32_t(best));
    }
  }
  uint64_t key[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = lane + 64 * i;
    const bool in = e < experts && (groups <= 1 || (kept >> (e / (experts / groups)) & 1));
    key[i] = in ? order_key(b[i], e) : 0;
  }
  float mine = 0.0f;      // lane j holds choice j
  int32_t my_id = 0;
  float sum = 0.0f;
  for (int j = 0; j < top_k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max_u64(best);
    const int e = static_cast<int>(0xffffffffu - uint32_t(best));
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (key[i] == best) {
        key[i] = 0;
        w = score[i];
      }
    }
    w = __shfl(w, e & 63);
    sum += w;
    if (lane == j) {
      mine = w;
      my_id = e;
    }
  }
  if (lane < top_k) {
    if (renorm) mine = mine / (sum + 1e-20f);
    ids[t * top_k + lane] = my_id;
    weights[t * top_k + lane] = mine * scale;
  }
}

// One wave a token.
template <int kN, bool kBf16, bool kSoftmax>
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ grad, const void* __restrict__ logits, int64_t tokens,
                                                             int experts, int64_t ld, const int32_t* __restrict__ ids, int top_k, bool renorm,
                                                             float scale, void* __restrict__ dlogits, int64_t ld_d) {
  const int lane = threadIdx.x & 63;
  const int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  // lane j < top_k holds choice j
  int id = -1;
  float g = 0.0f, w = 0.0f, rest = 0.0f;
  if (lane < top_k) {
    id = ids[t * top_k + lane];
    g = grad[t * top_k + lane] * scale;
  }
  const bool live = id >= 0 && id < experts;
  if (!live) { id = -1; g = 0.0f; }
  float s[kN];
  if constexpr (kSoftmax) {
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = lane + 64 * i;
      s[i] = e < experts ? load_logit<kBf16>(logits, t * ld + e) : kNegInf;
      top = fmaxf(top, s[i]);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      s[i] = expf(s[i] - top);
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] /= sum;
    if (live) w = expf(load_logit<kBf16>(logits, t * ld + id) - top) / sum;
  } else if (live) {
    const float x = load_logit<kBf16>(logits, t * ld + id);
    w = 1.0f / (1.0f + expf(-x));
    rest = 1.0f / (1.0f + expf(x));
  }
  if (renorm) {
    const float total = wave_sum(w) + 1e-20f;
    const float mean = wave_sum(g * (w / total));
    g = live ? (g - mean) / total : 0.0f;
  }
  const float gw = g * w;
  const float dot = kSoftmax ? wave_sum(gw) : 0.0f;
  const float add = kSoftmax ? gw : gw * rest;
  float d[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) d[i] = kSoftmax ? -s[i] * dot : 0.0f;
  for (int j = 0; j < top_k; ++j) {
    const int e = __shfl(id, j);
    const float a = __shfl(add, j);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (e == lane + 64 * i) d[i] += a;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = lane + 64 * i;
    if (e < experts) {
      if constexpr (kBf16) static_cast<__bf16*>(dlogits)[t * ld_d + e] = static_cast<__bf16>(d[i]);
      else static_cast<float*>(dlogits)[t * ld_d + e] = d[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Dispatch: a stable counting sort of the choices by expert, then the rows.
//
// The choices fall into chunks of kChunk.  A first kernel counts each chunk's
// experts into counts[chunk][expert]; a second one adds up the chunks before
// its own and the experts before each expert, ranks its own choices and
// writes order, position and offsets; a third quantizes each token's row
// once and writes it at its top_k places.
constexpr int kChunk = 1024;

__device__ __forceinline__ int choice_bin(const int32_t* ids, int64_t i, int experts) {
  const int32_t e = ids[i];
  return e >= 0 && e < experts ? e : experts;
}

__global__ __launch_bounds__(kChunk) void dispatch_count_kernel(const int32_t* __restrict__ ids, int64_t n, int experts,
                                                                int32_t* __restrict__ counts) {
  __shared__ int32_t bins[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= experts; e += kChunk) bins[e] = 0;
  __syncthreads();
  const int64_t i = int64_t(blockIdx.x) * kChunk + threadIdx.x;
  if (i < n) atomicAdd(&bins[choice_bin(ids, i, experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= experts; e += kChunk) counts[int64_t(blockIdx.x) * (experts + 1) + e] = bins[e];
}

__global__ __launch_bounds__(kChunk) void dispatch_rank_kernel(const int32_t* __restrict__ ids, int64_t n, int experts, int chunks,
                                                               const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ order, int32_t* __restrict__ position) {
  __shared__ int32_t base[kMaxExperts + 1], scan[kMaxExperts + 1];
  __shared__ int16_t mine[kChunk];
  const int chunk = blockIdx.x, tid = threadIdx.x;
  for (int e = tid; e <= experts; e += kChunk) {
    int before = 0, total = 0;
    for (int k = 0; k < chunks; ++k) {
      const int v = counts[int64_t(k) * (experts + 1) + e];
      if (k < chunk) before += v;
      total += v;
    }
    base[e] = before;
    scan[e] = total;
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    for (int e = 0; e <= experts; ++e) {
      const int total = scan[e];
      scan[e] = at;
      at += total;
    }
  }
  __syncthreads();
  if (chunk == 0)
    for (int e = tid; e <= experts; e += kChunk) offsets[e] = scan[e];
  const int64_t i = int64_t(chunk) * kChunk + tid;
  const int e = i < n ? choice_bin(ids, i, experts) : -1;
  mine[tid] = static_cast<int16_t>(e);
  __syncthreads();
  if (i < n) {
    int rank = 0;
    for (int k = 0; k < tid; ++k) rank += mine[k] == e;
    const int place = scan[e] + base[e] + rank;
    position[i] = place;
    order[place] = static_cast<int32_t>(i);
  }
}

// Workgroup (token, 2048 columns): lane of 8 columns, 16 lanes a tile.
template <bool kBf16>
__global__ __launch_bounds__(256) void dispatch_rows_kernel(const void* __restrict__ x, int64_t cols, int64_t ld_x, int top_k, int experts,
                                                            const int32_t* __restrict__ ids, const int32_t* __restrict__ position,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int64_t t = blockIdx.y;
  const int64_t col = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (col >= cols) return;
  float v[8];
  if constexpr (kBf16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + t * ld_x + col);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    const float* src = static_cast<const float*>(x) + t * ld_x + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = src[j];
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
  const float s = tile_scale(row16_max(amax));
  const u32x2 codes = {pack4_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s), pack4_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s)};
  for (int j = 0; j < top_k; ++j) {
    const int32_t e = ids[t * top_k + j];
    const int64_t place = position[t * top_k + j];
    const bool live = e >= 0 && e < experts;
    *reinterpret_cast<u32x2*>(q + place * cols + col) = live ? codes : u32x2{0, 0};
    if ((threadIdx.x & 15) == 0) scale[place * (cols / 128) + col / 128] = live ? s : 1.0f;
  }
}

fp8bs_status check_router(const char* fn, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld, int32_t top_k, int32_t score,
                          double scale) {
  if (!valid_dtype(dtype)) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (score != FP8BS_SCORE_SIGMOID && score != FP8BS_SCORE_SOFTMAX) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown score %d", fn, score);
  if (tokens < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (experts < 1 || experts > kMaxExperts)
    return fail(FP8BS_ERR_SHAPE, "%s: %lld experts, 1 to %d are supported", fn, (long long)experts, kMaxExperts);
  if (top_k < 1 || top_k > kMaxTopK) return fail(FP8BS_ERR_SHAPE, "%s: top_k %d is not in 1 .. %d", fn, top_k, kMaxTopK);
  if (ld < experts) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch smaller than the row", fn);
  if (!sane_matrix(tokens, ld, elem_size(dtype))) return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes and pitches exceed any allocation", fn);
  if (!std::isfinite(scale)) return fail(FP8BS_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  return FP8BS_OK;
}
bool aligned_elem(const void* p, int32_t dtype) { return reinterpret_cast<uintptr_t>(p) % elem_size(dtype) == 0; }

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

// One instantiation per number of experts a lane holds.
#define FP8BS_BY_EXPERTS(L) \
  do { \
    const int64_t per = (experts + 63) / 64; \
    if (per <= 1) L(1); \
    else if (per <= 2) L(2); \
    else if (per <= 4) L(4); \
    else if (per <= 8) L(8); \
    else L(16); \
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
  const dim3 grid(static_cast<uint32_t>((tokens + kRouteWaves - 1) / kRouteWaves));
  const bool bf16 = dtype == FP8BS_BF16, softmax = score == FP8BS_SCORE_SOFTMAX;
  begin_launch();
#define FP8BS_LL(N, B, S) hipLaunchKernelGGL((route_kernel<N, B, S>), grid, dim3(kRouteWaves * 64), 0, stream, logits, tokens, \
                                             static_cast<int>(experts), ld, bias, groups, top_groups, top_k, renormalize != 0, \
                                             static_cast<float>(scale), ids, weights)
#define FP8BS_L(N) \
  do { \
    if (bf16) { if (softmax) FP8BS_LL(N, true, true); else FP8BS_LL(N, true, false); } \
    else { if (softmax) FP8BS_LL(N, false, true); else FP8BS_LL(N, false, false); } \
  } while (0)
  FP8BS_BY_EXPERTS(FP8BS_L);
#undef FP8BS_L
#undef FP8BS_LL
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
  const dim3 grid(static_cast<uint32_t>((tokens + 3) / 4));
  const bool bf16 = dtype == FP8BS_BF16, softmax = score == FP8BS_SCORE_SOFTMAX;
  begin_launch();
#define FP8BS_LL(N, B, S) hipLaunchKernelGGL((route_backward_kernel<N, B, S>), grid, dim3(256), 0, stream, grad, logits, tokens, \
                                             static_cast<int>(experts), ld, ids, top_k, renormalize != 0, static_cast<float>(scale), \
                                             dlogits, ld_d)
#define FP8BS_L(N) \
  do { \
    if (bf16) { if (softmax) FP8BS_LL(N, true, true); else FP8BS_LL(N, true, false); } \
    else { if (softmax) FP8BS_LL(N, false, true); else FP8BS_LL(N, false, false); } \
  } while (0)
  FP8BS_BY_EXPERTS(FP8BS_L);
#undef FP8BS_L
#undef FP8BS_LL
  return check_launch(fn);
}

extern "C" int64_t fp8_moe_dispatch_workspace(int64_t tokens, int32_t experts, int32_t top_k) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || tokens >= (int64_t(1) << 31) / top_k) {
    fail(FP8BS_ERR_SHAPE, "fp8_moe_dispatch_workspace: sizes out of range");
    return -1;
  }
  return (tokens * top_k + kChunk - 1) / kChunk * (experts + 1) * 4;
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
  const int chunks = static_cast<int>((n + kChunk - 1) / kChunk);
  int32_t* counts = static_cast<int32_t*>(workspace);
  begin_launch();
  if (n) hipLaunchKernelGGL(dispatch_count_kernel, dim3(chunks), dim3(kChunk), 0, stream, ids, n, experts, counts);
  hipLaunchKernelGGL(dispatch_rank_kernel, dim3(std::max(chunks, 1)), dim3(kChunk), 0, stream, ids, n, experts, chunks, counts, offsets,
                     order, position);
  if (n) {
    for (int64_t t0 = 0; t0 < tokens; t0 += 65535) {
      const int64_t m = std::min<int64_t>(tokens - t0, 65535);
      const dim3 grid(static_cast<uint32_t>((cols + 2047) / 2048), static_cast<uint32_t>(m));
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

// Root-mean-square norm of rows and its gradient for gfx950.
//
//   h = x + residual (rounded to the rows' type), r = rsqrt(mean(h^2) + eps)
//   y = h r w, out in the rows' type and / or as E4M3 codes in 1x128 tiles
//   dx = r (g - h r^2 mean(g h)) + dresidual,  g = dy w
//   dw = sum over rows of dy h r
//
// Both are bound by memory: a row is read once, kept in registers from its
// sum to its outputs, and written once.  Up to kT threads share a row, 8 values
// (16 bytes of bf16) at kC places each; the 16 lanes of a DPP row hold one
// 1x128 tile at each place.  A worker (one wave, or one workgroup where a row
// needs more) walks rows with the weight in registers; neighbouring workers
// take neighbouring rows, so that the chip reads one region at a time.
#include <algorithm>

#include "fp8bs_train.h"
#include "rows.hpp"

namespace fp8bs {
namespace {

constexpr int64_t kMaxCols = 32768;

// Sums in 64 bits over the 16 lanes of a DPP row and the 64 of a wave, the same
// in every lane.
template <int kCtrl>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), kCtrl, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), kCtrl, 0xF, 0xF, false);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ double row16_sum(double v) {
  v += dpp_d<0x128>(v);
  v += dpp_d<0x124>(v);
  v += dpp_d<0x122>(v);
  return v + dpp_d<0x121>(v);
}
// v of neighbouring rows (k16) or of the wave's halves, added.
template <bool k16>
__device__ __forceinline__ double add_swapped(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(u), hi = static_cast<uint32_t>(u >> 32);
  const auto l = k16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false) : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto h = k16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false) : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return __builtin_bit_cast(double, uint64_t(h[0]) << 32 | l[0]) + __builtin_bit_cast(double, uint64_t(h[1]) << 32 | l[1]);
}
__device__ __forceinline__ double wave_sum(double v) { return add_swapped<false>(add_swapped<true>(row16_sum(v))); }

// Sums of the threads of a row, which has `waves` waves, in 64 bits: a thread's
// own 32 squares of at most 2^60 stay in float32's range, a wave's may not.  kT >
// 64: through LDS, `parity` alternating between calls, so that one barrier
// serves each.
template <int kT, int kN>
__device__ __forceinline__ void row_sum(const float (&v)[kN], double (&sum)[kN], double (*lds)[kN][16], int parity, int waves) {
#pragma unroll
  for (int n = 0; n < kN; ++n) sum[n] = wave_sum(static_cast<double>(v[n]));
  if constexpr (kT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < kN; ++n) lds[parity][n][wave] = sum[n];
    }
    __syncthreads();
    const int w = threadIdx.x & 15;           // at most 16 waves: one to a lane of a DPP row
#pragma unroll
    for (int n = 0; n < kN; ++n) sum[n] = row16_sum(w < waves ? lds[parity][n][w] : 0.0);
  }
}

// 1 / sqrt(m): the hardware's root, off by up to a unit in the last place, and
// one Newton step whose remainder is taken in 64 bits.  All values of a row
// share its error, and that of the mean: with both in float32, 2048 rows of 7168
// were off by 0.89 * 2^-24 (root mean square, no weight); elementary float32
// operations are off by 0.76, this by 0.64.  With the step's correction kept
// apart (0.44) more codes differ from those of the elementary operations, 10010
// in 117 million and not 3153, and as many from those of exact values: y / scale
// of bf16 rows and weights has no root in it, and one in 2400 lies on a border of
// two codes, where the order of the roundings decides.  A sum that is not finite
// gives NaN.
__device__ __forceinline__ float inverse_root(double m) {
  const float r = __builtin_amdgcn_rsqf(static_cast<float>(m));
  const double d = r;
  return __builtin_fmaf(0.5f * r, static_cast<float>(__builtin_fma(-m * d, d, 1.0)), r);
}

// This thread's weights (1 without a weight), anything past the row's end.
template <int kC>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int cols, int t, int threads, float (&out)[kC][8]) {
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int col = (c * threads + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) out[c][i] = 1.0f;
    if (w && col < cols) {
      if (bf16) widen<true>(load8<true, false>(at<true>(w, 0, 0, col)), out[c]);
      else widen<false>(load8<false, false>(at<false>(w, 0, 0, col)), out[c]);
    }
  }
}

// Values widened before this point are widened again behind it, not kept:
// twice the registers would halve the rows in flight.
template <bool kBf16, int kC>
__device__ __forceinline__ void keep_raw(Raw8<kBf16> (&r)[kC]) {
  if constexpr (kBf16) {
#pragma unroll
    for (int c = 0; c < kC; ++c) asm volatile("" : "+v"(r[c].u[0]));
  }
}

struct NormView {
  const void *x, *residual, *weight;
  void *residual_out, *y;
  uint8_t* q;
  float* scale;
  int64_t ld_x, ld_residual, ld_residual_out, ld_y, ld_q;
  double inv;                                 // 1 / cols
  int32_t rows, cols;
  float eps;
  int16_t threads;                            // of a row
  int16_t w_bf16;
};

// kResidual: with the residual's addition.  What is in the rows' type goes past
// the caches, the codes, which a GEMM reads next, through them: 16387 rows of
// 7168 take 169 us so, 196 with one of the two others through them too, 198 with
// both, 185 with nothing.
template <bool kBf16, int kT, int kC, bool kResidual>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void rmsnorm_kernel(const NormView a) {
  __shared__ double lds[2][1][16];
  const int t = kT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t worker = kT == 64 ? int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : blockIdx.x;
  const int64_t stride = int64_t(gridDim.x) * (kT == 64 ? 4 : 1);
  float w[kC][8];
  const int threads = kT == 64 ? 64 : a.threads;
  load_weight<kC>(a.weight, a.w_bf16, a.cols, t, threads, w);
  int parity = 0;
  for (int64_t row = worker; row < a.rows; row += stride, parity ^= 1) {
    Raw8<kBf16> h[kC], res[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) {
        h[c] = load8<kBf16>(at<kBf16>(a.x, row, a.ld_x, col));
        if constexpr (kResidual) res[c] = load8<kBf16>(at<kBf16>(a.residual, row, a.ld_residual, col));
      }
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) {
        float v[8];
        widen<kBf16>(h[c], v);
        if constexpr (kResidual) {
          float o[8];
          widen<kBf16>(res[c], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += o[i];
          h[c] = narrow<kBf16>(v);
          store8<kBf16, true>(at<kBf16>(a.residual_out, row, a.ld_residual_out, col), h[c]);
          widen<kBf16>(h[c], v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(v[i], v[i], sum[0]);
      }
    }
    double total[1];
    row_sum<kT, 1>(sum, total, lds, parity, threads >> 6);
    keep_raw<kBf16, kC>(h);
    const float r = inverse_root(__builtin_fma(total[0], a.inv, a.eps));
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) {
        float v[8];
        widen<kBf16>(h[c], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[c][i];
        if (a.y) store8<kBf16, true>(at<kBf16>(a.y, row, a.ld_y, col), narrow<kBf16>(v));
        if (a.q) {
          float s;
          const uint2 codes = quantize_tile(v, s);
          *reinterpret_cast<uint2*>(a.q + row * a.ld_q + static_cast<uint32_t>(col)) = codes;
          if ((t & 15) == 0) a.scale[row * (a.cols >> 7) + (col >> 7)] = s;
        }
      }
    }
  }
}

struct NormBackView {
  const void *dy, *h, *weight, *dresidual;
  void* dx;
  float* partial;                             // [workgroups, cols], the weight's gradient over each one's rows; NULL without
  int64_t ld_dy, ld_h, ld_dresidual, ld_dx;
  double inv;
  int32_t rows, cols;
  float eps;
  int16_t threads;
  int16_t w_bf16;
};

template <bool kBf16, int kT, int kC>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void rmsnorm_backward_kernel(const NormBackView a) {
  __shared__ double lds[2][2][16];
  const int t = kT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t worker = kT == 64 ? int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : blockIdx.x;
  const int64_t stride = int64_t(gridDim.x) * (kT == 64 ? 4 : 1);
  float w[kC][8], dw[kC][8];
  const int threads = kT == 64 ? 64 : a.threads;
  load_weight<kC>(a.weight, a.w_bf16, a.cols, t, threads, w);
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  int parity = 0;
  for (int64_t row = worker; row < a.rows; row += stride, parity ^= 1) {
    Raw8<kBf16> h[kC], g[kC], res[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) {
        h[c] = load8<kBf16>(at<kBf16>(a.h, row, a.ld_h, col));
        g[c] = load8<kBf16>(at<kBf16>(a.dy, row, a.ld_dy, col));
        if (a.dresidual) res[c] = load8<kBf16>(at<kBf16>(a.dresidual, row, a.ld_dresidual, col));
      }
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if ((c * threads + t) * 8 < a.cols) {
        float u[8], v[8];
        widen<kBf16>(h[c], u);
        widen<kBf16>(g[c], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] = __builtin_fmaf(u[i], u[i], sum[0]);
          sum[1] = __builtin_fmaf(v[i] * w[c][i], u[i], sum[1]);
        }
      }
    }
    double total[2];
    row_sum<kT, 2>(sum, total, lds, parity, threads >> 6);
    keep_raw<kBf16, kC>(h);
    keep_raw<kBf16, kC>(g);
    const float r = inverse_root(__builtin_fma(total[0], a.inv, a.eps));
    const float along = r * r * static_cast<float>(total[1] * a.inv);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) {
        float u[8], v[8], d[8];
        widen<kBf16>(h[c], u);
        widen<kBf16>(g[c], v);
        if (a.dresidual) widen<kBf16>(res[c], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[c][i] = __builtin_fmaf(v[i] * r, u[i], dw[c][i]);
          const float z = __builtin_fmaf(v[i], w[c][i], -u[i] * along);
          d[i] = a.dresidual ? __builtin_fmaf(r, z, d[i]) : r * z;
        }
        store8<kBf16>(at<kBf16>(a.dx, row, a.ld_dx, col), narrow<kBf16>(d));
      }
    }
  }
  if (!a.partial) return;
  float* const out = a.partial + int64_t(blockIdx.x) * a.cols;
  if constexpr (kT == 64) {                   // the four waves' sums join, in their order
    __shared__ float joined[2048];
    for (int k = 0; k < 4; ++k) {
      if (static_cast<int>(threadIdx.x >> 6) == k) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const int col = (c * 64 + t) * 8;
          if (col < a.cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) joined[col + i] = k ? joined[col + i] + dw[c][i] : dw[c][i];
          }
        }
      }
      __syncthreads();
    }
    for (int col = threadIdx.x * 4; col < a.cols; col += 1024) *reinterpret_cast<float4*>(out + col) = *reinterpret_cast<const float4*>(&joined[col]);
  } else {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * threads + t) * 8;
      if (col < a.cols) store8<false>(at<false>(out, 0, 0, col), narrow<false>(dw[c]));
    }
  }
}

// out[c] = sum over the workgroups of partial[workgroup][c]: 32 columns (one
// line) a workgroup, every 128th one's four columns in a thread.  None: zeros.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ partial, int n, int cols, float* __restrict__ out) {
  __shared__ float4 part[128][8];
  const int lane = threadIdx.x & 7, slot = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + lane * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int w = slot; w < n; w += 128) {
    const float4 p = *reinterpret_cast<const float4*>(partial + int64_t(w) * cols + col);
    s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
  }
  part[slot][lane] = s;
  __syncthreads();
  // Thread k * 32 + c joins column c of the slots k, k + 32, ..; then the 32.
  const float* p = reinterpret_cast<const float*>(part);
  float total = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) total += p[(threadIdx.x >> 5) * 32 + k * 1024 + (threadIdx.x & 31)];
  __syncthreads();
  float* const q = reinterpret_cast<float*>(part);
  q[threadIdx.x] = total;
  __syncthreads();
  if (threadIdx.x < 32) {
    total = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) total += q[32 * k + threadIdx.x];
    out[blockIdx.x * 32 + threadIdx.x] = total;
  }
}

// How rows are shared out: `threads` of a row (of at most `limit`) at `places`
// places each, in `blocks` workgroups.
struct Plan {
  int limit, threads, places;
  int64_t blocks;
  int workers() const { return threads == 64 ? 4 : 1; }          // of a workgroup
  uint32_t block() const { return static_cast<uint32_t>(threads * workers()); }
};
Plan make_plan(int64_t rows, int64_t cols) {
  Plan p;
  p.limit = cols <= 2048 ? 64 : (cols <= 8192 ? 512 : 1024);
  p.places = 1;
  while (int64_t(p.limit) * p.places * 8 < cols) p.places *= 2;
  p.threads = static_cast<int>((cols / 8 + p.places * 64 - 1) / (p.places * 64) * 64);
  p.blocks = (rows + p.workers() - 1) / p.workers();
  return p;
}
// A whole number of workgroups a CU, about 20 waves of them: 16387 rows of 7168
// (7 waves) take 190 us with two, 169 with three, 170 with four, 16384 of 4096 (8
// waves) 98, 99 and 98; numbers between leave CUs without work at the end (184
// and 109 with 3.4).
Plan forward_plan(int64_t rows, int64_t cols) {
  Plan p = make_plan(rows, cols);
  p.blocks = std::min<int64_t>(p.blocks, 256 * std::max(1u, std::min(4u, 21 * 64 / p.block())));
  return p;
}
// Two (one of 1024 threads): each leaves a row of sums behind, which the column
// sum has to read.  8195 rows of 7168 take 95 us with one, 83 with two, 93 with
// three, 88 with four; 8192 float32 rows of 2048 63, 61, 77 and 65; 1000 of 32768
// 97 with one and 112 with two.  No more of them than their largest share needs
// (513 rows of 16384 27 us otherwise, 23 so, 1062 of 7168 21.7 and 21.1), and two
// rows at least to a workgroup that works on one at a time (300 of 7168 13.3
// otherwise, 11.7 so; with waves that do, 704 of 1408, 9.9 so and 9.3 otherwise).
Plan backward_plan(int64_t rows, int64_t cols) {
  Plan p = make_plan(rows, cols);
  const int64_t most = 256 * (p.block() <= 512 ? 2 : 1);
  const int64_t each = std::max<int64_t>(p.workers() == 1 ? 2 : 1, (p.blocks + most - 1) / most);
  p.blocks = (p.blocks + each - 1) / each;
  return p;
}

// Calls f with the plan's constants.  A workgroup of 1024 threads leaves a thread
// 128 registers, which rows of more than 16384 columns pass: the gradient keeps
// 124 (bf16) and 272 (float32) bytes of scratch a thread there, the norm of
// float32 rows with a residual 52.
template <class F>
void with_plan(const Plan& p, F f) {
#define FP8BS_CASE(T, C) \
  if (p.limit == T && p.places == C) return f(std::integral_constant<int, T>{}, std::integral_constant<int, C>{})
  FP8BS_CASE(64, 1);
  FP8BS_CASE(64, 2);
  FP8BS_CASE(64, 4);
  FP8BS_CASE(512, 1);
  FP8BS_CASE(512, 2);
  FP8BS_CASE(1024, 2);
  FP8BS_CASE(1024, 4);
#undef FP8BS_CASE
}

fp8bs_status check_sizes(const char* fn, int64_t rows, int64_t cols, int64_t dtype, const void* weight, int64_t w_dtype, double eps) {
  if (rows < 0 || cols < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols == 0 || cols % 128 || cols > kMaxCols)
    return fail(FP8BS_ERR_SHAPE, "%s: cols=%lld must be a multiple of 128 in 128..%lld", fn, (long long)cols, (long long)kMaxCols);
  if ((dtype != FP8BS_BF16 && dtype != FP8BS_F32) || (weight && w_dtype != FP8BS_BF16 && w_dtype != FP8BS_F32))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown type %lld or %lld", fn, (long long)dtype, (long long)w_dtype);
  const float e = static_cast<float>(eps);
  if (!(e >= 0x1p-126f && e < __builtin_inff())) return fail(FP8BS_ERR_INVALID_ARG, "%s: eps must be a positive normal float32", fn);
  if (rows > kMaxExtent - 1) return fail(FP8BS_ERR_INVALID_ARG, "%s: rows=%lld exceed any allocation", fn, (long long)rows);
  if (weight && !aligned16(weight)) return fail(FP8BS_ERR_ALIGNMENT, "%s: weight must be 16-byte aligned", fn);
  return FP8BS_OK;
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" fp8bs_status fp8_rmsnorm_quant(const fp8bs_rmsnorm_args* args, hipStream_t stream) {
  const char* fn = "fp8_rmsnorm_quant";
  if (!args) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const fp8bs_rmsnorm_args& a = *args;
  if (fp8bs_status st = check_sizes(fn, a.rows, a.cols, a.dtype, a.weight, a.w_dtype, a.eps)) return st;
  if (a.rows == 0) return FP8BS_OK;
  if (!a.residual != !a.residual_out) return fail(FP8BS_ERR_INVALID_ARG, "%s: residual and residual_out come together", fn);
  if (!a.q != !a.scale) return fail(FP8BS_ERR_INVALID_ARG, "%s: q and scale come together", fn);
  if (!a.q && !a.y) return fail(FP8BS_ERR_INVALID_ARG, "%s: neither y nor q is asked for", fn);
  const int elt = elem_size(static_cast<int32_t>(a.dtype));
  if (fp8bs_status st = check_matrix(fn, "x", a.x, a.rows, a.cols, a.ld_x, elt)) return st;
  if (a.residual) {
    if (fp8bs_status st = check_matrix(fn, "residual", a.residual, a.rows, a.cols, a.ld_residual, elt)) return st;
    if (fp8bs_status st = check_matrix(fn, "residual_out", a.residual_out, a.rows, a.cols, a.ld_residual_out, elt)) return st;
  }
  if (a.y)
    if (fp8bs_status st = check_matrix(fn, "y", a.y, a.rows, a.cols, a.ld_y, elt)) return st;
  if (a.q) {
    if (fp8bs_status st = check_matrix(fn, "q", a.q, a.rows, a.cols, a.ld_q, 1)) return st;
    if (!aligned4(a.scale)) return fail(FP8BS_ERR_ALIGNMENT, "%s: scale must be 4-byte aligned", fn);
  }
  if (fp8bs_status st = check_apart(fn,
                                    {{"residual_out", matrix_block(a.residual_out, a.rows, a.cols, a.ld_residual_out, elt), true},
                                     {"y", matrix_block(a.y, a.rows, a.cols, a.ld_y, elt), true},
                                     {"q", matrix_block(a.q, a.rows, a.cols, a.ld_q, 1), false},
                                     {"scale", line(a.scale, a.rows * (a.cols / 128) * 4), false}},
                                    {{"x", matrix_block(a.x, a.rows, a.cols, a.ld_x, elt), true},
                                     {"residual", matrix_block(a.residual, a.rows, a.cols, a.ld_residual, elt), true},
                                     {"weight", line(a.weight, a.cols * elem_size(static_cast<int32_t>(a.w_dtype))), false}}))
    return st;
  const Plan p = forward_plan(a.rows, a.cols);
  const NormView v{a.x, a.residual, a.weight, a.residual_out, a.y, a.q, a.scale, a.ld_x, a.ld_residual, a.ld_residual_out, a.ld_y, a.ld_q,
                   1.0 / static_cast<double>(a.cols), static_cast<int32_t>(a.rows), static_cast<int32_t>(a.cols), static_cast<float>(a.eps),
                   static_cast<int16_t>(p.threads), a.w_dtype == FP8BS_BF16};
  begin_launch();
  with_plan(p, [&](auto threads, auto places) {
    constexpr int kT = decltype(threads)::value, kC = decltype(places)::value;
    const dim3 grid(static_cast<uint32_t>(p.blocks)), block(p.block());
    if (a.dtype == FP8BS_BF16) {
      if (a.residual) hipLaunchKernelGGL((rmsnorm_kernel<true, kT, kC, true>), grid, block, 0, stream, v);
      else hipLaunchKernelGGL((rmsnorm_kernel<true, kT, kC, false>), grid, block, 0, stream, v);
    } else {
      if (a.residual) hipLaunchKernelGGL((rmsnorm_kernel<false, kT, kC, true>), grid, block, 0, stream, v);
      else hipLaunchKernelGGL((rmsnorm_kernel<false, kT, kC, false>), grid, block, 0, stream, v);
    }
  });
  return check_launch(fn);
}

extern "C" int64_t fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxExtent - 1 || cols <= 0 || cols % 128 || cols > kMaxCols) return -1;
  const int64_t blocks = rows ? backward_plan(rows, cols).blocks : 0;
  return blocks > 1 ? blocks * cols * 4 : 0;
}

extern "C" fp8bs_status fp8_rmsnorm_backward(const fp8bs_rmsnorm_backward_args* args, hipStream_t stream) {
  const char* fn = "fp8_rmsnorm_backward";
  if (!args) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const fp8bs_rmsnorm_backward_args& a = *args;
  if (fp8bs_status st = check_sizes(fn, a.rows, a.cols, a.dtype, a.weight, a.w_dtype, a.eps)) return st;
  if (a.dweight && !aligned16(a.dweight)) return fail(FP8BS_ERR_ALIGNMENT, "%s: dweight must be 16-byte aligned", fn);
  const int cols = static_cast<int>(a.cols);
  const dim3 sum_grid(cols / 32), sum_block(1024);
  if (a.rows == 0) {
    if (!a.dweight) return FP8BS_OK;
    begin_launch();
    hipLaunchKernelGGL(column_sum_kernel, sum_grid, sum_block, 0, stream, nullptr, 0, cols, a.dweight);
    return check_launch(fn);
  }
  const int elt = elem_size(static_cast<int32_t>(a.dtype));
  if (fp8bs_status st = check_matrix(fn, "dy", a.dy, a.rows, a.cols, a.ld_dy, elt)) return st;
  if (fp8bs_status st = check_matrix(fn, "h", a.h, a.rows, a.cols, a.ld_h, elt)) return st;
  if (a.dresidual)
    if (fp8bs_status st = check_matrix(fn, "dresidual", a.dresidual, a.rows, a.cols, a.ld_dresidual, elt)) return st;
  if (fp8bs_status st = check_matrix(fn, "dx", a.dx, a.rows, a.cols, a.ld_dx, elt)) return st;
  const Plan p = backward_plan(a.rows, a.cols);
  float* partial = nullptr;
  const int64_t need = a.dweight ? fp8_rmsnorm_backward_workspace(a.rows, a.cols) : 0;
  if (a.dweight) {
    if (need > 0 && (!a.workspace || a.workspace_bytes < need))
      return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace of %lld bytes needed", fn, (long long)need);
    if (need > 0 && !aligned16(a.workspace)) return fail(FP8BS_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    partial = need > 0 ? static_cast<float*>(a.workspace) : a.dweight;      // one workgroup's sum is the result
  }
  if (fp8bs_status st = check_apart(fn,
                                    {{"dx", matrix_block(a.dx, a.rows, a.cols, a.ld_dx, elt), true},
                                     {"dweight", line(a.dweight, a.cols * 4), false},
                                     {"workspace", line(need > 0 ? a.workspace : nullptr, need), false}},
                                    {{"dy", matrix_block(a.dy, a.rows, a.cols, a.ld_dy, elt), true},
                                     {"h", matrix_block(a.h, a.rows, a.cols, a.ld_h, elt), true},
                                     {"dresidual", matrix_block(a.dresidual, a.rows, a.cols, a.ld_dresidual, elt), true},
                                     {"weight", line(a.weight, a.cols * elem_size(static_cast<int32_t>(a.w_dtype))), false}}))
    return st;
  const NormBackView v{a.dy, a.h, a.weight, a.dresidual, a.dx, partial, a.ld_dy, a.ld_h, a.ld_dresidual, a.ld_dx, 1.0 / static_cast<double>(a.cols),
                       static_cast<int32_t>(a.rows), cols, static_cast<float>(a.eps), static_cast<int16_t>(p.threads), a.w_dtype == FP8BS_BF16};
  begin_launch();
  with_plan(p, [&](auto threads, auto places) {
    constexpr int kT = decltype(threads)::value, kC = decltype(places)::value;
    const dim3 grid(static_cast<uint32_t>(p.blocks)), block(p.block());
    if (a.dtype == FP8BS_BF16) hipLaunchKernelGGL((rmsnorm_backward_kernel<true, kT, kC>), grid, block, 0, stream, v);
    else hipLaunchKernelGGL((rmsnorm_backward_kernel<false, kT, kC>), grid, block, 0, stream, v);
  });
  if (need > 0)
    hipLaunchKernelGGL(column_sum_kernel, sum_grid, sum_block, 0, stream, partial, static_cast<int>(p.blocks), cols, a.dweight);
  return check_launch(fn);
}

// Root-mean-square norm of rows and its gradient for gfx950.
//
//   h = x + residual (rounded to the rows' type), r = rsqrt(mean(h^2) + eps)
//   y = h r w, out in the rows' type and / or as E4M3 codes in 1x128 tiles
//   dx = r (g - h r^2 mean(g h)) + dresidual,  g = dy w
//   dw = sum over rows of dy h r
//
// Both are bound by memory: a row is read once, kept in registers from its
// sum to its outputs, and written once.  kT threads share a row, 8 values (16
// bytes of bf16) at kC places each, kT * 8 columns apart; the 16 lanes of a
// DPP row hold one 1x128 tile at each place.  A worker (one wave, or one
// workgroup where a row needs more) walks rows with the weight in registers.
#include <algorithm>

#include "fp8bs_train.h"
#include "rows.hpp"

namespace fp8bs {
namespace {

constexpr int64_t kMaxCols = 32768;

// Sums over the threads of a row.  kT > 64: through LDS, `parity` alternating
// between calls, so that one barrier serves each.
template <int kT, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*lds)[kN][16], int parity) {
#pragma unroll
  for (int n = 0; n < kN; ++n) v[n] = wave_sum(v[n]);
  if constexpr (kT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < kN; ++n) lds[parity][n][wave] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kT / 64; ++w) s += lds[parity][n][w];
      v[n] = s;
    }
  }
}

// This thread's weights (1 without a weight), 0 past the row's end.
template <int kT, int kC>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int cols, int t, float (&out)[kC][8]) {
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int col = (c * kT + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) out[c][i] = 1.0f;
    if (w && col < cols) {
      if (bf16) widen<true>(load8<true, false>(at<true>(w, 0, 0, col)), out[c]);
      else widen<false>(load8<false, false>(at<false>(w, 0, 0, col)), out[c]);
    }
  }
}

struct NormView {
  const void *x, *residual, *weight;
  void *residual_out, *y;
  uint8_t* q;
  float* scale;
  int64_t rows, per;                          // rows of a worker
  int64_t ld_x, ld_residual, ld_residual_out, ld_y, ld_q;
  int32_t cols;
  int32_t w_bf16;
  float eps;
};

template <bool kBf16, int kT, int kC>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void rmsnorm_kernel(const NormView a) {
  __shared__ float lds[2][1][16];
  const int t = kT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t worker = kT == 64 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t first = worker * a.per, last = min(first + a.per, a.rows);
  float w[kC][8];
  load_weight<kT, kC>(a.weight, a.w_bf16, a.cols, t, w);
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = first; row < last; ++row) {
    Raw8<kBf16> h[kC], res[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
      if (col < a.cols) {
        h[c] = load8<kBf16>(at<kBf16>(a.x, row, a.ld_x, col));
        if (a.residual) res[c] = load8<kBf16>(at<kBf16>(a.residual, row, a.ld_residual, col));
      }
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
      if (col < a.cols) {
        float v[8];
        widen<kBf16>(h[c], v);
        if (a.residual) {
          float o[8];
          widen<kBf16>(res[c], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += o[i];
          h[c] = narrow<kBf16>(v);
          store8<kBf16>(at<kBf16>(a.residual_out, row, a.ld_residual_out, col), h[c]);
          widen<kBf16>(h[c], v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(v[i], v[i], sum[0]);
      }
    }
    row_sum<kT, 1>(sum, lds, row & 1);
    const float r = rsqrtf(__builtin_fmaf(sum[0], inv, a.eps));
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
      if (col < a.cols) {
        float v[8];
        widen<kBf16>(h[c], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[c][i];
        if (a.y) store8<kBf16>(at<kBf16>(a.y, row, a.ld_y, col), narrow<kBf16>(v));
        if (a.q) {
          float s;
          const uint2 codes = quantize_tile(v, s);
          *reinterpret_cast<uint2*>(a.q + row * a.ld_q + col) = codes;
          if ((t & 15) == 0) a.scale[row * (a.cols >> 7) + (col >> 7)] = s;
        }
      }
    }
  }
}

struct NormBackView {
  const void *dy, *h, *weight, *dresidual;
  void* dx;
  float* partial;                             // [workers, cols], the weight's gradient over each worker's rows; NULL without
  int64_t rows, per;
  int64_t ld_dy, ld_h, ld_dresidual, ld_dx;
  int32_t cols;
  int32_t w_bf16;
  float eps;
};

template <bool kBf16, int kT, int kC>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void rmsnorm_backward_kernel(const NormBackView a) {
  __shared__ float lds[2][2][16];
  const int t = kT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t worker = kT == 64 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t first = worker * a.per, last = min(first + a.per, a.rows);
  if (first >= last) return;                  // a whole wave or workgroup
  float w[kC][8], dw[kC][8];
  load_weight<kT, kC>(a.weight, a.w_bf16, a.cols, t, w);
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  const float inv = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = first; row < last; ++row) {
    Raw8<kBf16> h[kC], g[kC], res[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
      if (col < a.cols) {
        h[c] = load8<kBf16>(at<kBf16>(a.h, row, a.ld_h, col));
        g[c] = load8<kBf16>(at<kBf16>(a.dy, row, a.ld_dy, col));
        if (a.dresidual) res[c] = load8<kBf16>(at<kBf16>(a.dresidual, row, a.ld_dresidual, col));
      }
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if ((c * kT + t) * 8 < a.cols) {
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
    row_sum<kT, 2>(sum, lds, row & 1);
    const float r = rsqrtf(__builtin_fmaf(sum[0], inv, a.eps));
    const float along = r * r * (sum[1] * inv);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
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
  if (a.partial) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int col = (c * kT + t) * 8;
      if (col < a.cols) store8<false>(at<false>(a.partial, worker, a.cols, col), narrow<false>(dw[c]));
    }
  }
}

// out[c] = sum over the workers of partial[worker][c]: 64 columns a workgroup,
// every 16th worker's four columns in a thread.  No workers: zeros.
__global__ __launch_bounds__(256) void column_sum_kernel(const float* __restrict__ partial, int workers, int cols, float* __restrict__ out) {
  __shared__ float4 part[16][16];
  const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + lane * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int w = slot; w < workers; w += 16) {
    const float4 p = *reinterpret_cast<const float4*>(partial + int64_t(w) * cols + col);
    s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
  }
  part[slot][lane] = s;
  __syncthreads();
  if (threadIdx.x < 64) {
    const float* p = reinterpret_cast<const float*>(part) + threadIdx.x;
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) total += p[64 * k];
    out[blockIdx.x * 64 + threadIdx.x] = total;
  }
}

// How rows are shared out: `threads` of a row at `places` places each, workers
// of `per` rows.
struct Plan {
  int threads, places;
  int64_t per, workers;
  uint32_t blocks() const { return static_cast<uint32_t>(threads == 64 ? (workers + 3) / 4 : workers); }
};
Plan make_plan(int64_t rows, int64_t cols, int64_t most_threads) {
  Plan p;
  p.threads = cols <= 2048 ? 64 : (cols <= 8192 ? 256 : 1024);
  p.places = 1;
  while (int64_t(p.threads) * p.places * 8 < cols) p.places *= 2;
  const int64_t most = most_threads / p.threads;
  p.per = std::max<int64_t>(1, (rows + most - 1) / most);
  p.workers = (rows + p.per - 1) / p.per;
  return p;
}
Plan forward_plan(int64_t rows, int64_t cols) { return make_plan(rows, cols, 256 * 5 * 256); }
Plan backward_plan(int64_t rows, int64_t cols) { return make_plan(rows, cols, 256 * 3 * 256); }

// Calls f with the plan's constants.
template <class F>
void with_plan(const Plan& p, F f) {
#define FP8BS_CASE(T, C) \
  if (p.threads == T && p.places == C) return f(std::integral_constant<int, T>{}, std::integral_constant<int, C>{})
  FP8BS_CASE(64, 1);
  FP8BS_CASE(64, 2);
  FP8BS_CASE(64, 4);
  FP8BS_CASE(256, 2);
  FP8BS_CASE(256, 4);
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
  const Plan p = forward_plan(a.rows, a.cols);
  const NormView v{a.x, a.residual, a.weight, a.residual_out, a.y, a.q, a.scale, a.rows, p.per, a.ld_x, a.ld_residual, a.ld_residual_out,
                   a.ld_y, a.ld_q, static_cast<int32_t>(a.cols), a.w_dtype == FP8BS_BF16, static_cast<float>(a.eps)};
  begin_launch();
  with_plan(p, [&](auto threads, auto places) {
    constexpr int kT = decltype(threads)::value, kC = decltype(places)::value;
    const dim3 grid(p.blocks()), block(kT < 256 ? 256 : kT);
    if (a.dtype == FP8BS_BF16) hipLaunchKernelGGL((rmsnorm_kernel<true, kT, kC>), grid, block, 0, stream, v);
    else hipLaunchKernelGGL((rmsnorm_kernel<false, kT, kC>), grid, block, 0, stream, v);
  });
  return check_launch(fn);
}

extern "C" int64_t fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxExtent - 1 || cols <= 0 || cols % 128 || cols > kMaxCols) return -1;
  const int64_t workers = rows ? backward_plan(rows, cols).workers : 0;
  return workers > 1 ? workers * cols * 4 : 0;
}

extern "C" fp8bs_status fp8_rmsnorm_backward(const fp8bs_rmsnorm_backward_args* args, hipStream_t stream) {
  const char* fn = "fp8_rmsnorm_backward";
  if (!args) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const fp8bs_rmsnorm_backward_args& a = *args;
  if (fp8bs_status st = check_sizes(fn, a.rows, a.cols, a.dtype, a.weight, a.w_dtype, a.eps)) return st;
  if (a.dweight && !aligned16(a.dweight)) return fail(FP8BS_ERR_ALIGNMENT, "%s: dweight must be 16-byte aligned", fn);
  const int cols = static_cast<int>(a.cols);
  const dim3 sum_grid(cols / 64), sum_block(256);
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
  if (a.dweight) {
    const int64_t need = fp8_rmsnorm_backward_workspace(a.rows, a.cols);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need))
      return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace of %lld bytes needed", fn, (long long)need);
    if (need > 0 && !aligned16(a.workspace)) return fail(FP8BS_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
    partial = need > 0 ? static_cast<float*>(a.workspace) : a.dweight;      // one worker's sum is the result
  }
  const NormBackView v{a.dy, a.h, a.weight, a.dresidual, a.dx, partial, a.rows, p.per, a.ld_dy, a.ld_h, a.ld_dresidual, a.ld_dx, cols,
                       a.w_dtype == FP8BS_BF16, static_cast<float>(a.eps)};
  begin_launch();
  with_plan(p, [&](auto threads, auto places) {
    constexpr int kT = decltype(threads)::value, kC = decltype(places)::value;
    const dim3 grid(p.blocks()), block(kT < 256 ? 256 : kT);
    if (a.dtype == FP8BS_BF16) hipLaunchKernelGGL((rmsnorm_backward_kernel<true, kT, kC>), grid, block, 0, stream, v);
    else hipLaunchKernelGGL((rmsnorm_backward_kernel<false, kT, kC>), grid, block, 0, stream, v);
  });
  if (partial != a.dweight)
    hipLaunchKernelGGL(column_sum_kernel, sum_grid, sum_block, 0, stream, partial, static_cast<int>(p.workers), cols, a.dweight);
  return check_launch(fn);
}

// Gated activation between an expert's two GEMMs, and its gradient, for
// gfx950.  With s = sigmoid(g):
//   y  = g s u
//   dg = dy u s (1 + g (1 - s)),   du = dy g s
// out in the rows' type and / or as E4M3 codes in 1x128 tiles.
//
// Bound by memory: every value is read once and every output written once.
// The 16 lanes of a DPP row hold one 1x128 tile, 8 values each; a wave takes
// 4 tiles a step and kU steps, all loads issued before the first use.  What is
// in the rows' type goes past the caches, the codes, which a GEMM reads next,
// through them: the gradient of 32768 x 2048 takes 124 us so, 140 the other way
// round, 141 with all through them, 133 with nothing.
#include "fp8bs_train.h"
#include "rows.hpp"

namespace fp8bs {
namespace {

// silu(g) = g sigmoid(g) = g / (1 + e), e = exp(-g), as q + c: a quotient by the
// hardware's reciprocal and its remainder's.  e is 2^n times the hardware's exp2
// of at most 1/2 (the argument's remainder is taken with log2(e) in two parts):
// adding 1.5 * 2^23 leaves the rounded n in the low bits, which go into the
// exponent.  At gates beyond 87 on either side e is that of 87; below -87
// silu counts as 0.
// Roundings: exp2, 1 + e, the result (q by itself where a gradient needs silu
// as one value).  32768 x 2048 in bf16 with codes: 74 us, rms error 0.80 * 2^-24
// (elementary float32 operations 0.82); with exp(-|g|), which needs selections
// and a product more, 75 and 0.84.
struct Gate {
  float q, c;
  float slope;                                // of silu: s (1 + g (1 - s)) = s + silu (1 - s)
  __device__ __forceinline__ float silu() const { return q + c; }
  // silu * v, rounded once.
  __device__ __forceinline__ float times(float v) const { return __builtin_fmaf(c, v, q * v); }
};
template <bool kSlope>
__device__ __forceinline__ Gate gate(float g) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kEdge = 87.0f, kRound = 0x1.8p23f;
  const float x = __builtin_amdgcn_fmed3f(g, -kEdge, kEdge);
  const float n = __builtin_fmaf(x, -kLog2e, kRound);
  const float part = __builtin_fmaf(x, -kLog2eLow, __builtin_fmaf(x, -kLog2e, -(n - kRound)));
  const float e = __uint_as_float(__float_as_uint(__builtin_amdgcn_exp2f(part)) + (__float_as_uint(n) << 23));
  const float d = 1.0f + e;
  const float r = g < -kEdge ? 0.0f : __builtin_amdgcn_rcpf(d);
  Gate z{};
  z.q = g * r;
  z.c = __builtin_fmaf(-z.q, d, g) * r;
  if constexpr (kSlope) {
    const float s = __builtin_fmaf(-__builtin_fmaf(d, r, -1.0f), r, r);
    z.slope = __builtin_fmaf(fminf(z.silu(), kEdge), e * s, s);
  }
  return z;
}

struct ActView {
  const void *dy, *gate, *up;
  void* y;                                    // d in the backward pass
  uint8_t* q;
  float* scale;
  int64_t ld_dy, ld_gate, ld_up, ld_y, ld_q;
  FastDiv per_row;                            // tiles in a row of gate
  uint32_t tiles;
};

template <bool kBf16, int kU>
__global__ __launch_bounds__(256) void swiglu_kernel(const ActView a) {
  const int lane = threadIdx.x & 63;
  const uint32_t tile0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (4 * kU) + (lane >> 4);
  Raw8<kBf16> g[kU], u[kU];
  uint32_t row[kU], block[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const uint32_t t = tile0 + 4 * k;
    row[k] = a.per_row.div(t);
    block[k] = t - row[k] * a.per_row.d;
    if (t < a.tiles) {
      const int col = block[k] * 128 + (lane & 15) * 8;
      g[k] = load8<kBf16>(at<kBf16>(a.gate, row[k], a.ld_gate, col));
      u[k] = load8<kBf16>(at<kBf16>(a.up, row[k], a.ld_up, col));
    }
  }
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    if (tile0 + 4 * k >= a.tiles) break;
    const int col = block[k] * 128 + (lane & 15) * 8;
    float x[8], v[8];
    widen<kBf16>(g[k], x);
    widen<kBf16>(u[k], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = gate<false>(x[i]).times(v[i]);    // no larger than x on the way: gate * up could overflow
    if (a.y) store8<kBf16, true>(at<kBf16>(a.y, row[k], a.ld_y, col), narrow<kBf16>(v));
    if (a.q) {
      float s;
      const uint2 codes = quantize_tile(v, s);
      *reinterpret_cast<uint2*>(a.q + row[k] * a.ld_q + col) = codes;
      if ((lane & 15) == 0) a.scale[tile0 + 4 * k] = s;
    }
  }
}

template <bool kBf16, int kU>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const ActView a) {
  const int lane = threadIdx.x & 63;
  const uint32_t tile0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (4 * kU) + (lane >> 4);
  const int64_t cols = int64_t(a.per_row.d) * 128;
  Raw8<kBf16> dy[kU], g[kU], u[kU];
  uint32_t row[kU], block[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const uint32_t t = tile0 + 4 * k;
    row[k] = a.per_row.div(t);
    block[k] = t - row[k] * a.per_row.d;
    if (t < a.tiles) {
      const int col = block[k] * 128 + (lane & 15) * 8;
      dy[k] = load8<kBf16>(at<kBf16>(a.dy, row[k], a.ld_dy, col));
      g[k] = load8<kBf16>(at<kBf16>(a.gate, row[k], a.ld_gate, col));
      u[k] = load8<kBf16>(at<kBf16>(a.up, row[k], a.ld_up, col));
    }
  }
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    if (tile0 + 4 * k >= a.tiles) break;
    float d[8], x[8], v[8];
    widen<kBf16>(dy[k], d);
    widen<kBf16>(g[k], x);
    widen<kBf16>(u[k], v);
    float out[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Gate z = gate<true>(x[i]);
      out[0][i] = z.slope * d[i] * v[i];
      out[1][i] = z.silu() * d[i];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t col = h * cols + block[k] * 128 + (lane & 15) * 8;
      if (a.y) store8<kBf16, true>(at<kBf16>(a.y, row[k], a.ld_y, 0) + col * (kBf16 ? 2 : 4), narrow<kBf16>(out[h]));
      if (a.q) {
        float s;
        const uint2 codes = quantize_tile(out[h], s);
        *reinterpret_cast<uint2*>(a.q + row[k] * a.ld_q + col) = codes;
        if ((lane & 15) == 0) a.scale[(int64_t(row[k]) * 2 + h) * a.per_row.d + block[k]] = s;
      }
    }
  }
}

// Steps a wave takes: with fewer than this many tiles, one, so that more
// workgroups share them.
constexpr int64_t kFewTiles = 256 * 4 * 4 * 8;

fp8bs_status check_sizes(const char* fn, int64_t rows, int64_t cols, int64_t dtype) {
  if (rows < 0 || cols < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (cols % 128) return fail(FP8BS_ERR_SHAPE, "%s: cols=%lld must be a multiple of 128", fn, (long long)cols);
  if (dtype != FP8BS_BF16 && dtype != FP8BS_F32) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown type %lld", fn, (long long)dtype);
  // Tiles: a launch has fewer than 2^32 threads, and takes 32 tiles with 256.
  if (rows > kMaxExtent - 1 || cols > kMaxExtent / 4 || rows * (cols / 128) > (int64_t(1) << 29) - 64)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: %lld x %lld exceed any allocation", fn, (long long)rows, (long long)cols);
  return FP8BS_OK;
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

#define FP8BS_LAUNCH_ACT(KERNEL)                                                                                     \
  {                                                                                                                  \
    const int steps = tiles < kFewTiles ? 1 : 2;                                                                     \
    const dim3 grid(static_cast<uint32_t>((tiles + 16 * steps - 1) / (16 * steps))), block(256);                     \
    begin_launch();                                                                                                  \
    if (a.dtype == FP8BS_BF16) {                                                                                     \
      if (steps == 1) hipLaunchKernelGGL((KERNEL<true, 1>), grid, block, 0, stream, v);                              \
      else hipLaunchKernelGGL((KERNEL<true, 2>), grid, block, 0, stream, v);                                         \
    } else {                                                                                                         \
      if (steps == 1) hipLaunchKernelGGL((KERNEL<false, 1>), grid, block, 0, stream, v);                             \
      else hipLaunchKernelGGL((KERNEL<false, 2>), grid, block, 0, stream, v);                                        \
    }                                                                                                                \
    return check_launch(fn);                                                                                         \
  }

extern "C" fp8bs_status fp8_swiglu_quant(const fp8bs_swiglu_args* args, hipStream_t stream) {
  const char* fn = "fp8_swiglu_quant";
  if (!args) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const fp8bs_swiglu_args& a = *args;
  if (fp8bs_status st = check_sizes(fn, a.rows, a.cols, a.dtype)) return st;
  if (a.rows == 0 || a.cols == 0) return FP8BS_OK;
  if (!a.q != !a.scale) return fail(FP8BS_ERR_INVALID_ARG, "%s: q and scale come together", fn);
  if (!a.q && !a.y) return fail(FP8BS_ERR_INVALID_ARG, "%s: neither y nor q is asked for", fn);
  const int elt = elem_size(static_cast<int32_t>(a.dtype));
  if (fp8bs_status st = check_matrix(fn, "gate", a.gate, a.rows, a.cols, a.ld_gate, elt)) return st;
  if (fp8bs_status st = check_matrix(fn, "up", a.up, a.rows, a.cols, a.ld_up, elt)) return st;
  if (a.y)
    if (fp8bs_status st = check_matrix(fn, "y", a.y, a.rows, a.cols, a.ld_y, elt)) return st;
  if (a.q) {
    if (fp8bs_status st = check_matrix(fn, "q", a.q, a.rows, a.cols, a.ld_q, 1)) return st;
    if (!aligned4(a.scale)) return fail(FP8BS_ERR_ALIGNMENT, "%s: scale must be 4-byte aligned", fn);
  }
  if (fp8bs_status st = check_apart(fn,
                                    {{"y", matrix_block(a.y, a.rows, a.cols, a.ld_y, elt), true},
                                     {"q", matrix_block(a.q, a.rows, a.cols, a.ld_q, 1), false},
                                     {"scale", line(a.scale, a.rows * (a.cols / 128) * 4), false}},
                                    {{"gate", matrix_block(a.gate, a.rows, a.cols, a.ld_gate, elt), true},
                                     {"up", matrix_block(a.up, a.rows, a.cols, a.ld_up, elt), true}}))
    return st;
  const int64_t tiles = a.rows * (a.cols / 128);
  const ActView v{nullptr, a.gate, a.up, a.y, a.q, a.scale, 0, a.ld_gate, a.ld_up, a.ld_y, a.ld_q,
                  FastDiv(static_cast<uint32_t>(a.cols / 128)), static_cast<uint32_t>(tiles)};
  FP8BS_LAUNCH_ACT(swiglu_kernel)
}

extern "C" fp8bs_status fp8_swiglu_backward(const fp8bs_swiglu_backward_args* args, hipStream_t stream) {
  const char* fn = "fp8_swiglu_backward";
  if (!args) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const fp8bs_swiglu_backward_args& a = *args;
  if (fp8bs_status st = check_sizes(fn, a.rows, a.cols, a.dtype)) return st;
  if (a.rows == 0 || a.cols == 0) return FP8BS_OK;
  if (!a.q != !a.scale) return fail(FP8BS_ERR_INVALID_ARG, "%s: q and scale come together", fn);
  if (!a.q && !a.d) return fail(FP8BS_ERR_INVALID_ARG, "%s: neither d nor q is asked for", fn);
  const int elt = elem_size(static_cast<int32_t>(a.dtype));
  if (fp8bs_status st = check_matrix(fn, "dy", a.dy, a.rows, a.cols, a.ld_dy, elt)) return st;
  if (fp8bs_status st = check_matrix(fn, "gate", a.gate, a.rows, a.cols, a.ld_gate, elt)) return st;
  if (fp8bs_status st = check_matrix(fn, "up", a.up, a.rows, a.cols, a.ld_up, elt)) return st;
  if (a.d)
    if (fp8bs_status st = check_matrix(fn, "d", a.d, a.rows, 2 * a.cols, a.ld_d, elt)) return st;
  if (a.q) {
    if (fp8bs_status st = check_matrix(fn, "q", a.q, a.rows, 2 * a.cols, a.ld_q, 1)) return st;
    if (!aligned4(a.scale)) return fail(FP8BS_ERR_ALIGNMENT, "%s: scale must be 4-byte aligned", fn);
  }
  const void* const right = a.d ? static_cast<const char*>(a.d) + a.cols * elt : nullptr;
  if (fp8bs_status st = check_apart(fn,
                                    {{"d", matrix_block(a.d, a.rows, a.cols, a.ld_d, elt), true},
                                     {"d's right half", matrix_block(right, a.rows, a.cols, a.ld_d, elt), true},
                                     {"q", matrix_block(a.q, a.rows, 2 * a.cols, a.ld_q, 1), false},
                                     {"scale", line(a.scale, a.rows * (a.cols / 128) * 8), false}},
                                    {{"dy", matrix_block(a.dy, a.rows, a.cols, a.ld_dy, elt), true},
                                     {"gate", matrix_block(a.gate, a.rows, a.cols, a.ld_gate, elt), true},
                                     {"up", matrix_block(a.up, a.rows, a.cols, a.ld_up, elt), true}}))
    return st;
  const int64_t tiles = a.rows * (a.cols / 128);
  const ActView v{a.dy, a.gate, a.up, a.d, a.q, a.scale, a.ld_dy, a.ld_gate, a.ld_up, a.ld_d, a.ld_q,
                  FastDiv(static_cast<uint32_t>(a.cols / 128)), static_cast<uint32_t>(tiles)};
  FP8BS_LAUNCH_ACT(swiglu_backward_kernel)
}

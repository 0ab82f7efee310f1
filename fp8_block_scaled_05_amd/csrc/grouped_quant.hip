// Operands of the experts' weight gradients for gfx950: rows, gathered into
// the order of their experts, transposed and quantized in 128x1 tiles that
// start anew at every expert, with power-of-two scales.
//
// Bound by memory: 2 (or 4) bytes read and 1 written a value.  A workgroup
// takes 128 places of one expert and walks a strip of columns, 128 at a time.
// A thread loads 8 consecutive places at 8 consecutive columns (16-byte loads
// of bf16, 16 lanes on 256 consecutive bytes of a row), so that an 8x8
// transposition of bytes in registers leaves 8 consecutive codes of a column;
// through LDS they leave as whole 128-byte lines.
#include <algorithm>

#include "fp8bs_train.h"
#include "groups.hpp"
#include "rows.hpp"

namespace fp8bs {
namespace {

constexpr int kMinExp = -100;                 // the smallest exponent of a scale
constexpr int64_t kMaxColumns = int64_t(1) << 22;

struct View {
  const void* x;
  const int32_t *off, *order;
  uint8_t* q;
  float* scale;
  int32_t* padded;
  int64_t ld_x, ld_q;
  FastDiv top_k;
  int32_t rows, places, cols, G;
  int32_t scale_cols;                         // columns / 128
  int32_t blocks, strips, per_strip;          // workgroups: blocks of 128 places x strips of per_strip * 128 columns
};

// padded[0 .. G], by one wave.
__device__ __forceinline__ void write_padded(const View& a, int lane) {
  int run = 0, total = 0;
  if (lane == 0) a.padded[0] = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const GroupRange r = group_ranges(a.off, a.G, a.places, g0, lane, run);
    const int upto = prefix_sum((r.hi - r.lo + 127) >> 7, lane);
    if (g0 + lane < a.G) a.padded[g0 + lane + 1] = (total + upto) << 7;
    total += __shfl(upto, 63);
  }
}

// The places of block `b`: [lo, hi), or false if no expert has so many.
__device__ __forceinline__ bool find_block(const View& a, int b, int lane, int& lo, int& hi) {
  int run = 0, skip = b;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const GroupRange r = group_ranges(a.off, a.G, a.places, g0, lane, run);
    const int count = (r.hi - r.lo + 127) >> 7, upto = prefix_sum(count, lane);
    const uint64_t hit = __ballot(skip < upto);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int from = skip - (__shfl(upto, l) - __shfl(count, l));
      lo = __builtin_amdgcn_readfirstlane(__shfl(r.lo, l) + from * 128);
      hi = __builtin_amdgcn_readfirstlane(min(__shfl(r.hi, l), lo + 128));
      return true;
    }
    skip -= __shfl(upto, 63);
  }
  return false;
}

// 2^e of a tile: the smallest e >= kMinExp with amax <= 448 * 2^e (448 is
// 0.875 * 2^9: the carry into the exponent tells mantissas above 0.75), 0 for
// a tile of zeros.
__device__ __forceinline__ int tile_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int((u + 0x1fffffu) >> 23) - 135;
  return u == 0 ? 0 : max(e, kMinExp);
}
__device__ __forceinline__ float exp2_of(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// w[i] = bytes of row i (columns 0 .. 3 of one half) -> w[j] = bytes of column j (rows 0 .. 3).
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);   // r0c0 r1c0 r0c1 r1c1
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);   // r0c2 r1c2 r0c3 r1c3
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

template <bool kBf16>
__global__ __launch_bounds__(256) void grouped_t_kernel(const View a) {
  __shared__ __align__(16) float most[2][4][128];
  __shared__ __align__(16) uint8_t tile[128 * 128];   // [column][place], 16-byte chunks swizzled by the column
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // The hardware hands workgroup i to XCD i % 8: each XCD takes a contiguous
  // range of the walk, blocks first, so that the scales of neighbouring blocks
  // (4 bytes each, in one line) meet in its L2.
  const uint32_t n = gridDim.x, per = n >> 3, rest = n & 7u, xcd = blockIdx.x & 7u;
  const uint32_t id = xcd * per + min(xcd, rest) + (blockIdx.x >> 3);
  if (id == 0 && wave == 0) write_padded(a, lane);
  const int block = static_cast<int>(id % a.blocks), strip = static_cast<int>(id / a.blocks);
  int lo, hi;
  if (!find_block(a, block, lane, lo, hi)) return;

  const int cc = (t & 15) * 8, r0 = (t >> 4) * 8;
  int32_t source[8];                          // rows of x, -1: zeros
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = lo + r0 + i;
    source[i] = -1;
    if (p < hi) {
      if (a.order) {
        const uint32_t o = static_cast<uint32_t>(a.order[p]);
        const uint32_t row = a.top_k.div(o);
        source[i] = o <= 0x7fffffffu && row < static_cast<uint32_t>(a.rows) ? static_cast<int32_t>(row) : -1;
      } else {
        source[i] = p;
      }
    }
  }
  const int first = strip * a.per_strip * 128, last = min(first + a.per_strip * 128, a.cols);
  int parity = 0;
  for (int c0 = first; c0 < last; c0 += 128, parity ^= 1) {
    const int col = c0 + cc;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (source[i] >= 0 && col < a.cols) {
        widen<kBf16>(load8<kBf16, false>(at<kBf16>(a.x, source[i], a.ld_x, col)), v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
    }
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = fabsf(v[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m[j] = fmaxf(m[j], fabsf(v[i][j]));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 16));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 32));
    }
    if (lane < 16) {
      float4* d = reinterpret_cast<float4*>(&most[parity][wave][cc]);
      d[0] = make_float4(m[0], m[1], m[2], m[3]);
      d[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();                          // also: the last round's lines have left the tile
    float back[8];                            // 2^-e of this thread's columns
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 f = *reinterpret_cast<const float4*>(&most[parity][0][cc + 4 * h]);
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float4 g = *reinterpret_cast<const float4*>(&most[parity][w][cc + 4 * h]);
        f = make_float4(fmaxf(f.x, g.x), fmaxf(f.y, g.y), fmaxf(f.z, g.z), fmaxf(f.w, g.w));
      }
      back[4 * h] = f.x, back[4 * h + 1] = f.y, back[4 * h + 2] = f.z, back[4 * h + 3] = f.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = tile_exponent(back[j]);
      back[j] = exp2_of(-e);
      if (r0 == 0 && col < a.cols) a.scale[int64_t(col + j) * a.scale_cols + block] = exp2_of(e);
    }
    uint32_t code[2][8];                      // [column half][row]
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        code[h][i] = pack4_e4m3(v[i][4 * h] * back[4 * h], v[i][4 * h + 1] * back[4 * h + 1], v[i][4 * h + 2] * back[4 * h + 2],
                                v[i][4 * h + 3] * back[4 * h + 3]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t low[4] = {code[h][0], code[h][1], code[h][2], code[h][3]}, high[4] = {code[h][4], code[h][5], code[h][6], code[h][7]};
      transpose4(low);
      transpose4(high);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = cc + 4 * h + j;
        *reinterpret_cast<uint2*>(&tile[c * 128 + (((r0 >> 4) ^ ((c >> 3) & 7)) << 4) + (r0 & 8)]) = make_uint2(low[j], high[j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = (t >> 3) + 32 * k, chunk = t & 7;
      if (c0 + c < a.cols)
        *reinterpret_cast<uint4*>(a.q + (c0 + c) * a.ld_q + int64_t(block) * 128 + chunk * 16) =
            *reinterpret_cast<const uint4*>(&tile[c * 128 + ((chunk ^ ((c >> 3) & 7)) << 4)]);
    }
  }
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" int64_t fp8_quant_grouped_t_columns(int64_t places, int32_t G) {
  if (places < 0 || places > kMaxExtent - 1 || G < 1 || G > 1024) return -1;
  // A tile has at least one place, and every expert's last one may be short.
  return (places + 127 * std::min<int64_t>(places, G)) / 128 * 128;
}

extern "C" fp8bs_status fp8_quant_grouped_t(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const int32_t* off,
                                            int32_t G, const int32_t* order, int64_t places, int32_t top_k, uint8_t* q, int64_t ld_q,
                                            float* scale, int64_t columns, int32_t* padded, hipStream_t stream) {
  const char* fn = "fp8_quant_grouped_t";
  if (rows < 0 || cols < 0 || places < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (G < 1 || G > 1024) return fail(FP8BS_ERR_INVALID_ARG, "%s: G=%d outside 1..1024", fn, G);
  if (!valid_dtype(x_dtype)) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown x_dtype %d", fn, x_dtype);
  if (cols % 16) return fail(FP8BS_ERR_SHAPE, "%s: cols=%lld must be a multiple of 16", fn, (long long)cols);
  if (top_k < 1 || top_k > 1024) return fail(FP8BS_ERR_INVALID_ARG, "%s: top_k=%d outside 1..1024", fn, top_k);
  if (rows > kMaxExtent - 1 || places > kMaxExtent - 1 || cols > kMaxExtent - 256)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes exceed any allocation", fn);
  if (!order && (places != rows || top_k != 1))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: without order places must be rows and top_k 1", fn);
  const int64_t need = fp8_quant_grouped_t_columns(places, G);
  if (columns % 128 || columns < need)
    return fail(FP8BS_ERR_SHAPE, "%s: columns=%lld must be a multiple of 128 and at least %lld", fn, (long long)columns, (long long)need);
  if (columns > kMaxColumns) return fail(FP8BS_ERR_INVALID_ARG, "%s: columns=%lld above 2^22", fn, (long long)columns);
  if (!off || !padded) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned4(off) || !aligned4(padded) || !aligned4(order)) return fail(FP8BS_ERR_ALIGNMENT, "%s: index arrays must be 4-byte aligned", fn);
  const bool work = places > 0 && cols > 0;
  if (work) {
    if (rows > 0)
      if (fp8bs_status st = check_matrix(fn, "x", x, rows, cols, ld_x, elem_size(x_dtype))) return st;
    if (fp8bs_status st = check_matrix(fn, "q", q, cols, columns, ld_q, 1)) return st;
    if (!scale) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (scale)", fn);
    if (!aligned4(scale)) return fail(FP8BS_ERR_ALIGNMENT, "%s: scale must be 4-byte aligned", fn);
  }
  View v{x, off, order, q, scale, padded, ld_x, ld_q, FastDiv(static_cast<uint32_t>(top_k)), static_cast<int32_t>(rows),
         static_cast<int32_t>(places), static_cast<int32_t>(cols), G, static_cast<int32_t>(columns / 128), 1, 1, 0};
  if (work) {
    // Strips of as many columns as leave about 2048 workgroups: a workgroup
    // looks its places up once.
    const int64_t blocks = need / 128, wide = (cols + 127) / 128;
    const int64_t strips = std::min(wide, (2048 + blocks - 1) / blocks);
    v.blocks = static_cast<int32_t>(blocks);
    v.per_strip = static_cast<int32_t>((wide + strips - 1) / strips);
    v.strips = static_cast<int32_t>((wide + v.per_strip - 1) / v.per_strip);
  }
  const dim3 grid(static_cast<uint32_t>(v.blocks) * v.strips), block(256);
  begin_launch();
  if (x_dtype == FP8BS_BF16) hipLaunchKernelGGL(grouped_t_kernel<true>, grid, block, 0, stream, v);
  else hipLaunchKernelGGL(grouped_t_kernel<false>, grid, block, 0, stream, v);
  return check_launch(fn);
}

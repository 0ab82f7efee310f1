// Operands of the experts' weight gradients for gfx950: rows, gathered into
// the order of their experts, transposed and quantized in 128x1 tiles that
// start anew at every expert, with power-of-two scales.
//
// Bound by memory: 2 (or 4) bytes read and 1 written a value.  A workgroup
// takes 128 places of one expert and walks a strip of columns, 128 at a time.
// A thread loads 8 consecutive places at 8 consecutive columns (16-byte loads of
// bf16, 16 lanes on 256 consecutive bytes of a row).  The converting instruction applies a tile's power of two and
// takes a column's values in pairs of places, so that 8 consecutive codes of a
// column come out in order; through LDS they leave as whole 128-byte lines.
#include <algorithm>

#include "fp8bs_train.h"
#include "groups.hpp"
#include "rows.hpp"

namespace fp8bs {
namespace {

constexpr int kMinExp = -100;                 // the smallest exponent of a scale
constexpr int kTopExp = 120;                  // that of the largest float32; codes there end at 240
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

// Codes of 256 and -256 (0x78 and 0xf8 of a word's bytes) as 240 and -240: 256 *
// 2^120 is beyond float32 and bf16.
__device__ __forceinline__ uint32_t at_most_240(uint32_t w) {
  const uint32_t other = (w & 0x7f7f7f7fu) ^ 0x78787878u;          // 0 where a byte is one
  return w - ((~(other + 0x7f7f7f7fu) & 0x80808080u) >> 7);
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// What the threads of a column exchange: for float32 the largest magnitudes of
// 8 columns; for bf16 the same as bits, two columns a word (the order of
// magnitudes is that of their bits).
template <bool kBf16>
struct Most {
  static constexpr int kWords = kBf16 ? 4 : 8;
  uint32_t w[kWords];
  __device__ __forceinline__ void join(int k, uint32_t v) {
    if constexpr (kBf16) {
      w[k] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, w[k]), __builtin_bit_cast(u16x2, v)));
    } else {
      w[k] = __float_as_uint(fmaxf(__uint_as_float(w[k]), __uint_as_float(v)));
    }
  }
  __device__ __forceinline__ float column(int j) const {
    if constexpr (kBf16) return (j & 1) ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
    else return __uint_as_float(w[j]);
  }
  // The largest of the 8 columns.
  __device__ __forceinline__ float all() const {
    Most m{{w[0]}};
#pragma unroll
    for (int k = 1; k < kWords; ++k) m.join(0, w[k]);
    return kBf16 ? fmaxf(m.column(0), m.column(1)) : m.column(0);
  }
};

// Word k of a thread's row.
template <bool kBf16>
__device__ __forceinline__ uint32_t word(const Raw8<kBf16>& r, int k) {
  return r.u[k / 4][k % 4];
}

// Codes of column j of rows i .. i + 3, from the raw rows, divided by s = 2^e.
template <bool kBf16>
__device__ __forceinline__ uint32_t encode4(const Raw8<kBf16> (&row)[8], int i, int j, float s) {
  i16x2 c = {0, 0};
  if constexpr (kBf16) {
    const uint32_t pick = (j & 1) ? 0x07060302u : 0x05040100u;      // one column's values of two rows
    const bf16x2 a = __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(word<true>(row[i + 1], j / 2), word<true>(row[i], j / 2), pick));
    const bf16x2 b = __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(word<true>(row[i + 3], j / 2), word<true>(row[i + 2], j / 2), pick));
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, a, s, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, b, s, true);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, __uint_as_float(word<false>(row[i], j)), __uint_as_float(word<false>(row[i + 1], j)), s, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, __uint_as_float(word<false>(row[i + 2], j)), __uint_as_float(word<false>(row[i + 3], j)), s, true);
  }
  return __builtin_bit_cast(uint32_t, c);
}

template <bool kBf16>
__global__ __launch_bounds__(256, kBf16 ? 4 : 3) void grouped_t_kernel(const View a) {
  using M = Most<kBf16>;
  __shared__ __align__(16) uint32_t most[2][4][16 * M::kWords];
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
  Raw8<kBf16> row[8];
  auto load = [&](int col) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      row[i] = Raw8<kBf16>{};
      if (source[i] >= 0 && col < last) row[i] = load8<kBf16, false>(at<kBf16>(a.x, source[i], a.ld_x, col));
    }
  };
  load(first + cc);
  int parity = 0;
  for (int c0 = first; c0 < last; c0 += 128, parity ^= 1) {
    const int col = c0 + cc;
    M m;
#pragma unroll
    for (int k = 0; k < M::kWords; ++k) {
      constexpr uint32_t kMagnitude = kBf16 ? 0x7fff7fffu : 0x7fffffffu;
      m.w[k] = word<kBf16>(row[0], k) & kMagnitude;
#pragma unroll
      for (int i = 1; i < 8; ++i) m.join(k, word<kBf16>(row[i], k) & kMagnitude);
      m.join(k, __shfl_xor(m.w[k], 16));
      m.join(k, __shfl_xor(m.w[k], 32));
    }
    u32x4* const mine = reinterpret_cast<u32x4*>(&most[parity][0][(t & 15) * M::kWords]);
    constexpr int kApart = 4 * M::kWords;     // 16-byte pieces between the waves'
    if (lane < 16) {
#pragma unroll
      for (int k = 0; k < M::kWords / 4; ++k) mine[wave * kApart + k] = u32x4{m.w[4 * k], m.w[4 * k + 1], m.w[4 * k + 2], m.w[4 * k + 3]};
    }
    __syncthreads();                          // also: the last round's lines have left the tile
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int k = 0; k < M::kWords / 4; ++k) {
        const u32x4 v = mine[w * kApart + k];
#pragma unroll
        for (int i = 0; i < 4; ++i) m.join(4 * k + i, v[i]);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = exp2_of(tile_exponent(m.column(j)));
      if (r0 == 0 && col < a.cols) a.scale[int64_t(col + j) * a.scale_cols + block] = s;
      const int c = cc + j;
      *reinterpret_cast<uint2*>(&tile[c * 128 + (((r0 >> 4) ^ ((c >> 3) & 7)) << 4) + (r0 & 8)]) =
          make_uint2(encode4<kBf16>(row, 0, j, s), encode4<kBf16>(row, 4, j, s));
    }
    if (__any(m.all() > 448.0f * exp2_of(kTopExp - 1))) {          // hardly ever: a look at this thread's own codes
      for (int c = cc; c < cc + 8; ++c) {
        uint2* const codes = reinterpret_cast<uint2*>(&tile[c * 128 + (((r0 >> 4) ^ ((c >> 3) & 7)) << 4) + (r0 & 8)]);
        if (m.column(c - cc) > 448.0f * exp2_of(kTopExp - 1)) *codes = make_uint2(at_most_240(codes->x), at_most_240(codes->y));
      }
    }
    load(col + 128);                          // the next columns' loads are in flight while these leave
    __syncthreads();
    // Stores past the caches: ordinary ones push the strip's rows out of the L2
    // (107 us where these take 63).
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = (t >> 3) + 32 * k, chunk = t & 7;
      if (c0 + c < a.cols)
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(&tile[c * 128 + ((chunk ^ ((c >> 3) & 7)) << 4)]),
                                    reinterpret_cast<u32x4*>(a.q + (c0 + c) * a.ld_q + int64_t(block) * 128 + chunk * 16));
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
  if (rows > kMaxExtent - 1 || places > kMaxExtent - 1 || cols > kMaxExtent / 4)
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
  if (fp8bs_status st = check_apart(fn,
                                    {{"padded", line(padded, (G + int64_t(1)) * 4), false},
                                     {"q", work ? matrix_block(q, cols, columns, ld_q, 1) : Block{}, false},
                                     {"scale", work ? line(scale, cols * (columns / 128) * 4) : Block{}, false}},
                                    {{"off", line(off, (G + int64_t(1)) * 4), false},
                                     {"order", line(order, places * 4), false},
                                     {"x", work ? matrix_block(x, rows, cols, ld_x, elem_size(x_dtype)) : Block{}, false}}))
    return st;
  View v{x, off, order, q, scale, padded, ld_x, ld_q, FastDiv(static_cast<uint32_t>(top_k)), static_cast<int32_t>(rows),
         static_cast<int32_t>(places), static_cast<int32_t>(cols), G, static_cast<int32_t>(columns / 128), 1, 1, 0};
  if (work) {
    // Strips of as many columns as leave about 4096 workgroups.  A workgroup
    // looks its places up once, but while all blocks of a strip are worked on,
    // gathered rows are read again from the L2 only if the strip's part of x
    // fits there: 32768 gathered rows of 7168 take 74 us with 2048 workgroups,
    // 63 with 4096, 64 with 8192, 75 with 16384.
    const int64_t blocks = need / 128, wide = (cols + 127) / 128;
    const int64_t strips = std::min(wide, (4096 + blocks - 1) / blocks);
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

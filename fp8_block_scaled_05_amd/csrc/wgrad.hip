// The experts' weight gradients for gfx950:
//   y[g] (+)= sum over expert g's own 128-deep blocks of A_block B_block^T,
// A [N, columns] and B [K, columns] E4M3 codes with one power-of-two scale per
// row and block.
//
// The scales are powers of two, so the instruction that widens E4M3 to bf16
// (v_cvt_scalef32_pk_bf16_fp8) applies them, exactly: the matrix cores'
// float32 accumulators are the result, with no promotion per block and no
// second set of registers for it.  What that leaves free goes into the wave's
// tile.  One of 128 x 64 widens 24 operand pieces for every 32 matrix
// instructions of 32x32x16, where one of 64 x 64 widens 16 for 16.
//
// Structure: a step's rows of kDeep bytes lie in LDS with their 16-byte chunks
// swizzled (see Cfg::off), two stages, filled by direct global-to-LDS loads one
// step ahead; scales come four blocks at a time.  Experts differ in depth: the
// tiles of each expert are shared out over all XCDs, so that a deep one does
// not keep a single XCD busy.
#include <algorithm>

#include "fp8bs_train.h"
#include "lds_dma.hpp"
#include "rows.hpp"

namespace fp8bs {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 w8 __attribute__((ext_vector_type(8)));

struct Args {
  const uint8_t *a, *b;
  const float *a_scale, *b_scale;
  const int32_t* padded;
  void* y;
  int64_t lda, ldb;
  int32_t N, K, blocks, G;                    // blocks: columns / 128
  int32_t tiles_n, tiles_k;                   // tiles of one expert
  int32_t tiles, share;                       // their product; workgroups of one expert (>= tiles)
  int32_t accumulate;
};

template <int BM_, int BN_, int WM_, int WN_, int kDeep_, int kShared_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int kDeep = kDeep_;        // of a step: a block or half of one
  static constexpr int kShared = kShared_;    // workgroups of a CU
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int TM = BM / WM, TN = BN / WN, SM = TM / 32, SN = TN / 32;
  static constexpr int kHalves = 128 / kDeep, kSlices = kDeep / 32, kRowsLoaded = 1024 / kDeep;
  static constexpr int kWalk = 4;             // height of the tile walk
  static_assert(BM % (kRowsLoaded * kWaves) == 0 && BN % (kRowsLoaded * kWaves) == 0 && BM % (16 * kWaves) == 0 && BN % (16 * kWaves) == 0 &&
                    (kRowsLoaded * kWaves) % 16 == 0,
                "loads must split evenly");
  // 16-byte chunk swizzle of a row, which repeats every 16 rows: that many
  // consecutive rows of one chunk fill all 64 banks once.
  static __device__ __forceinline__ int swizzle(int row) { return kDeep == 128 ? swz(row) : (row >> 2) & 3; }
  // Byte offset of logical chunk `chunk` of LDS row `row`.
  static __device__ __forceinline__ int off(int row, int chunk) { return row * kDeep + ((chunk ^ swizzle(row)) << 4); }
};

// 8 codes, scaled, as bf16 (exact).
__device__ __forceinline__ w8 widen8(uint32_t w0, uint32_t w1, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
  return w8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// kNT: y's values go past the caches.
template <class C, bool kBf16, bool kNT>
__global__ __launch_bounds__(C::kThreads, C::kShared) void wgrad_kernel(const Args args) {
  constexpr int SM = C::SM, SN = C::SN, NW = C::kWaves, kDeep = C::kDeep, kRL = C::kRowsLoaded;
  constexpr int kStage = (C::BM + C::BN) * kDeep;
  __shared__ __align__(16) uint8_t stage[2][kStage];             // A's rows, then B's
  __shared__ __align__(16) float scales[2][C::BM + C::BN][4];    // of four consecutive blocks
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Tile: workgroup i runs on XCD i % 8.  Each XCD takes a contiguous range of
  // every expert's tile walk, kWalk tiles of N high.
  const int g = blockIdx.x / args.share;
  int id = blockIdx.x % args.share;
  if (args.share >= 8) {
    const int x = id & 7, per = args.tiles >> 3, rest = args.tiles & 7;
    if ((id >> 3) >= per + (x < rest)) return;
    id = x * per + min(x, rest) + (id >> 3);
  }
  const int high = id / (C::kWalk * args.tiles_k), in = id - high * (C::kWalk * args.tiles_k);
  const int height = min(args.tiles_n - high * C::kWalk, C::kWalk);
  const int n0 = (high * C::kWalk + in % height) * C::BM, k0 = in / height * C::BN;
  const int rows = min(args.N - n0, C::BM), cols = min(args.K - k0, C::BN);

  // The expert's blocks: [first, first + depth).
  const int first = min(max(args.padded[g] >> 7, 0), args.blocks);
  const int depth = min(max(args.padded[g + 1] >> 7, first), args.blocks) - first;

  // Loads.  The hardware checks a raw buffer load's VGPR offset alone, so
  // every row-dependent part of an address is in the descriptor's base or in
  // that offset; the step's place in the row goes into the SGPR offset, which
  // stays inside any row that passes the check.  Load v of a wave covers rows
  // kRL (v NW + wave) and on, kRL of them; rows past the matrix read as zero.
  constexpr int LA = C::BM / kRL / NW, LB = C::BN / kRL / NW, SA = C::BM / 16 / NW, SB = C::BN / 16 / NW;
  const int lrow = kRL * wave + lane / (kDeep / 16);
  const int chunk = ((lane & (kDeep / 16 - 1)) ^ C::swizzle(lrow)) << 4;
  const int voff_a = lrow * int(args.lda) + chunk, voff_b = lrow * int(args.ldb) + chunk;
  const int voff_s = ((16 * wave + (lane >> 2)) * args.blocks + (lane & 3)) * 4;
  // An operand's descriptor: its base is the tile's first row at the expert's
  // first block, its size counts the rows that exist.
  auto describe = [](const void* base, int64_t row0, int64_t n, int64_t pitch, int64_t start) {
    return make_rsrc(static_cast<const uint8_t*>(base) + row0 * pitch + start, n * pitch - start);
  };
  const i32x4 rs_a = describe(args.a, n0, rows, args.lda, int64_t(first) * 128);
  const i32x4 rs_b = describe(args.b, k0, cols, args.ldb, int64_t(first) * 128);
  const i32x4 rs_sa = describe(args.a_scale, n0, rows, int64_t(args.blocks) * 4, int64_t(first) * 4);
  const i32x4 rs_sb = describe(args.b_scale, k0, cols, int64_t(args.blocks) * 4, int64_t(first) * 4);
  const int step_a = kRL * NW * int(args.lda), step_b = kRL * NW * int(args.ldb), step_s = 16 * NW * 4 * args.blocks;
  auto load_stage = [&](int s, int h) {
#pragma unroll
    for (int v = 0; v < LA; ++v) dma16(rs_a, lds_addr(&stage[s][(v * NW + wave) * 1024]), voff_a + v * step_a, h * kDeep);
#pragma unroll
    for (int v = 0; v < LB; ++v) dma16(rs_b, lds_addr(&stage[s][C::BM * kDeep + (v * NW + wave) * 1024]), voff_b + v * step_b, h * kDeep);
  };
  // Blocks 4 q .. 4 q + 3 into scales[q & 1].  A lane whose block is past the
  // expert's last reads another block's or the next row's scale (unused), or
  // zero behind the last row.
  auto load_scales = [&](int q) {
    const int vo = voff_s + q * 16;
#pragma unroll
    for (int u = 0; u < SA; ++u) dma4(rs_sa, lds_addr(&scales[q & 1][16 * (u * NW + wave)][0]), vo + u * step_s, 0);
#pragma unroll
    for (int u = 0; u < SB; ++u) dma4(rs_sb, lds_addr(&scales[q & 1][C::BM + 16 * (u * NW + wave)][0]), vo + u * step_s, 0);
  };

  const int wm = wave / C::WN, wn = wave % C::WN, r32 = lane & 31, hk = lane >> 5;
  const int arow = wm * C::TM + r32, brow = wn * C::TN + r32;
  int a_off[C::kSlices], b_off[C::kSlices];   // this lane's chunks of its first rows; 32 rows on they lie 32 kDeep bytes further
#pragma unroll
  for (int q = 0; q < C::kSlices; ++q) {
    a_off[q] = C::off(arow, C::kSlices * hk + q);
    b_off[q] = C::BM * kDeep + C::off(brow, C::kSlices * hk + q);
  }
  v16f acc[SM][SN];
#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int j = 0; j < SN; ++j) acc[i][j] = v16f{};

  uint4 ra[2][SM], rb[2][SN];
  float sa[2][SM], sb[2][SN];
  // Scales that are no power of two from 2^-100 to 2^120: `wide` exceeds the
  // range's width or `bits` has mantissa bits.  Thread t looks at row t's four
  // of a group; rows past the matrix and blocks past the expert's do not count.
  constexpr uint32_t kLow = uint32_t(127 - 100) << 23, kWidth = uint32_t(220) << 23;
  uint32_t wide = 0, bits = 0;
  auto check = [&](int kb) {
#pragma unroll
    for (int row = threadIdx.x; row < C::BM + C::BN; row += C::kThreads) {
      const bool real = row < C::BM ? row < rows : row - C::BM < cols;
      const float4 s = *reinterpret_cast<const float4*>(&scales[(kb >> 2) & 1][row][0]);
      const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t d = real && kb + k < depth ? __float_as_uint(v[k]) - kLow : 0u;
        wide = max(wide, d);
        bits |= d;
      }
    }
  };
  auto read_slice = [&](int s, int q, int buf) {
#pragma unroll
    for (int i = 0; i < SM; ++i) ra[buf][i] = *reinterpret_cast<const uint4*>(&stage[s][a_off[q] + 32 * kDeep * i]);
#pragma unroll
    for (int j = 0; j < SN; ++j) rb[buf][j] = *reinterpret_cast<const uint4*>(&stage[s][b_off[q] + 32 * kDeep * j]);
  };
  auto read_scales = [&](int kb, int buf) {
#pragma unroll
    for (int i = 0; i < SM; ++i) sa[buf][i] = scales[(kb >> 2) & 1][arow + 32 * i][kb & 3];
#pragma unroll
    for (int j = 0; j < SN; ++j) sb[buf][j] = scales[(kb >> 2) & 1][C::BM + brow + 32 * j][kb & 3];
  };
  auto multiply = [&](int buf, int sbuf) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      w8 fa[SM], fb[SN];
#pragma unroll
      for (int i = 0; i < SM; ++i)
        fa[i] = t ? widen8(ra[buf][i].z, ra[buf][i].w, sa[sbuf][i]) : widen8(ra[buf][i].x, ra[buf][i].y, sa[sbuf][i]);
#pragma unroll
      for (int j = 0; j < SN; ++j)
        fb[j] = t ? widen8(rb[buf][j].z, rb[buf][j].w, sb[sbuf][j]) : widen8(rb[buf][j].x, rb[buf][j].y, sb[sbuf][j]);
#pragma unroll
      for (int i = 0; i < SM; ++i)
#pragma unroll
        for (int j = 0; j < SN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  };
  // Step h (part h % kHalves of block kb) from stage s = h & 1; the next one, if
  // there is one, becomes visible at the barrier, which every read of stage s
  // precedes: the step after it is loaded there at once, and has a whole step
  // to arrive.  A group of scales is loaded with the first step that needs it;
  // its buffer held the group before the last, whose reads precede an earlier
  // barrier.
  const int steps = depth * C::kHalves;
  auto step = [&](auto s_c, auto p_c, int h) {
    constexpr int s = decltype(s_c)::value, p = decltype(p_c)::value;
    if (h % (4 * C::kHalves) == 0) check(h / C::kHalves);
#pragma unroll
    for (int q = 0; q + 1 < C::kSlices; ++q) {
      read_slice(s, q + 1, (q + 1) & 1);
      multiply(q & 1, p);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (h + 1 < steps) {
      wait_and_barrier<0>();
      if (h + 2 < steps) {
        load_stage(s, h + 2);
        if ((h + 2) % (4 * C::kHalves) == 0) load_scales((h + 2) / (4 * C::kHalves));
      }
      read_slice(s ^ 1, 0, 0);
      if (C::kHalves == 1 || s == 1) read_scales((h + 1) / C::kHalves, p ^ 1);
    }
    multiply(1, p);
    __builtin_amdgcn_sched_barrier(0);
  };

  if (depth > 0) {
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    load_scales(0);
    load_stage(0, 0);
    if (steps > 1) {
      load_stage(1, 1);
      wait_and_barrier<LA + LB>();
    } else {
      wait_and_barrier<0>();
    }
    read_slice(0, 0, 0);
    read_scales(0, 0);
    for (int h = 0; h < steps; h += 2 * C::kHalves) {
      if constexpr (C::kHalves == 1) {
        step(I0{}, I0{}, h);
        if (h + 1 < steps) step(I1{}, I1{}, h + 1);
      } else {
        step(I0{}, I0{}, h);
        step(I1{}, I0{}, h + 1);
        if (h + 2 < steps) {
          step(I0{}, I1{}, h + 2);
          step(I1{}, I1{}, h + 3);
        }
      }
    }
  } else if (args.accumulate) {
    return;
  }
  // Each wave's verdict on the scales that it saw.
  __shared__ int verdict[NW];
  const bool bad = __any(wide > kWidth || (bits & 0x7fffffu));
  if (lane == 0) verdict[wave] = bad;
  __syncthreads();
  bool broken = false;
#pragma unroll
  for (int w = 0; w < NW; ++w) broken |= verdict[w] != 0;

  // Accumulator r of subtile (i, j) is row wm TM + 32 i + 8 (r / 4) + 4 hk +
  // r % 4 and column wn TN + 32 j + r32: 32 lanes on consecutive columns, so a
  // float32 store fills whole 128-byte lines without LDS.  For bf16 two lanes
  // exchange values, and each stores two columns of one of two rows.  A row's
  // address is uniform but for hk.  Accumulating waits for each old value by
  // itself: 16 experts of 4096 x 7168 in float32, 2048 deep, take 3.0 ms, and 1.6
  // without, where the old values' bytes are 0.4.
  constexpr int kElt = kBf16 ? 2 : 4;
  const int pitch = args.K * kElt;
  char* const y = static_cast<char*>(args.y) + ((int64_t(g) * args.N + n0 + wm * C::TM) * args.K + k0 + wn * C::TN) * kElt;
  const int odd = kBf16 ? lane & 1 : 0, left = kBf16 ? r32 & ~1 : r32;
  const uint32_t voff = uint32_t(4 * hk + odd) * uint32_t(pitch) + uint32_t(left * kElt);
  const int rows_left = rows - wm * C::TM - 4 * hk - odd, cols_left = cols - wn * C::TN - left;
#pragma unroll
  for (int i = 0; i < SM; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += kBf16 ? 2 : 1) {
      const int row = 32 * i + 8 * (r >> 2) + (r & 3);
      char* const line = y + int64_t(row) * pitch;
#pragma unroll
      for (int j = 0; j < SN; ++j) {
        char* const p = line + (voff + 32 * j * kElt);
        const bool real = row < rows_left && 32 * j < cols_left;
        const float v0 = broken ? __builtin_nanf("") : acc[i][j][r];
        if constexpr (kBf16) {
          const float v1 = broken ? __builtin_nanf("") : acc[i][j][r + 1];
          const float other = __shfl_xor(odd ? v0 : v1, 1);
          float lo = odd ? other : v0, hi = odd ? v1 : other;
          if (real) {
            if (args.accumulate) {
              const uint32_t was = *reinterpret_cast<const uint32_t*>(p);
              lo += bf16_lo(was);
              hi += bf16_hi(was);
            }
            if constexpr (kNT) __builtin_nontemporal_store(round_bf16x2(lo, hi), reinterpret_cast<uint32_t*>(p));
            else *reinterpret_cast<uint32_t*>(p) = round_bf16x2(lo, hi);
          }
        } else if (real) {
          float* const f = reinterpret_cast<float*>(p);
          const float w = args.accumulate ? v0 + *f : v0;
          if constexpr (kNT) __builtin_nontemporal_store(w, f);
          else *f = w;
        }
      }
    }
}

using Large = Cfg<256, 256, 2, 4, 128, 1>;    // 8 waves of 128 x 64
// Tiles of 128 (4 waves of 64 x 64) and 64 (4 of 32 x 32), in steps of whole and
// of half blocks.  Half128 with float32 out keeps 8 bytes of scratch a thread.
using Whole128 = Cfg<128, 128, 2, 2, 128, 2>;
using Half128 = Cfg<128, 128, 2, 2, 64, 3>;
using Whole64 = Cfg<64, 64, 2, 2, 128, 4>;
using Half64 = Cfg<64, 64, 2, 2, 64, 4>;

template <class C>
fp8bs_status launch(Args args, bool bf16, hipStream_t stream) {
  const char* fn = "fp8_blockscaled_grouped_wgrad";
  args.tiles_n = (args.N + C::BM - 1) / C::BM;
  args.tiles_k = (args.K + C::BN - 1) / C::BN;
  const int64_t tiles = int64_t(args.tiles_n) * args.tiles_k, share = tiles < 8 ? tiles : (tiles + 7) / 8 * 8;
  if (share * args.G > 0xffffffffll / C::kThreads) return fail(FP8BS_ERR_INVALID_ARG, "%s: too many tiles", fn);
  args.tiles = static_cast<int32_t>(tiles);
  args.share = static_cast<int32_t>(share);
  const dim3 grid(static_cast<uint32_t>(share * args.G)), block(C::kThreads);
  // Past the caches where y's rows are whole lines and the experts shallow: 64
  // experts of 2048 x 2048 over 8192 rows take 210 us so and 269 otherwise, 16 of
  // 4096 x 7168 over 4096 rows 456 and 550, over 8192 rows 714 and 727, over 32768
  // 1709 and 1693.  Where two rows share a line it has to be read again: 32
  // experts of 512 x 1040 in bf16 take 22 us past the caches and 16 through them.
  const bool lines = int64_t(args.K) * (bf16 ? 2 : 4) % 128 == 0 && args.blocks <= 8 * args.G && !args.accumulate;
  begin_launch();
  if (bf16) {
    if (lines) hipLaunchKernelGGL((wgrad_kernel<C, true, true>), grid, block, 0, stream, args);
    else hipLaunchKernelGGL((wgrad_kernel<C, true, false>), grid, block, 0, stream, args);
  } else {
    if (lines) hipLaunchKernelGGL((wgrad_kernel<C, false, true>), grid, block, 0, stream, args);
    else hipLaunchKernelGGL((wgrad_kernel<C, false, false>), grid, block, 0, stream, args);
  }
  return check_launch(fn);
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" fp8bs_status fp8_blockscaled_grouped_wgrad(int64_t N, int64_t K, int64_t columns, int32_t G, const int32_t* padded,
                                                      const uint8_t* a, int64_t lda, const float* a_scale, const uint8_t* b, int64_t ldb,
                                                      const float* b_scale, void* y, int32_t y_dtype, int32_t accumulate,
                                                      hipStream_t stream) {
  const char* fn = "fp8_blockscaled_grouped_wgrad";
  if (N < 0 || K < 0 || columns < 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: negative size", fn);
  if (G < 1 || G > 1024) return fail(FP8BS_ERR_INVALID_ARG, "%s: G=%d outside 1..1024", fn, G);
  if (!valid_dtype(y_dtype)) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown y_dtype %d", fn, y_dtype);
  if (accumulate != 0 && accumulate != 1) return fail(FP8BS_ERR_INVALID_ARG, "%s: accumulate is %d", fn, accumulate);
  if (N % 16 || K % 16) return fail(FP8BS_ERR_SHAPE, "%s: N=%lld and K=%lld must be multiples of 16", fn, (long long)N, (long long)K);
  if (columns % 128) return fail(FP8BS_ERR_SHAPE, "%s: columns=%lld must be a multiple of 128", fn, (long long)columns);
  if (N == 0 || K == 0) return FP8BS_OK;
  const int64_t kWide = int64_t(1) << 22;
  if (columns > kWide || N > (int64_t(1) << 26) || K > (int64_t(1) << 26) || !sane_matrix(G * N, K, elem_size(y_dtype)))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: sizes exceed any allocation", fn);
  if (!padded || !y) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned4(padded)) return fail(FP8BS_ERR_ALIGNMENT, "%s: padded must be 4-byte aligned", fn);
  if (!aligned16(y)) return fail(FP8BS_ERR_ALIGNMENT, "%s: y must be 16-byte aligned", fn);
  if (columns > 0) {
    if (fp8bs_status st = check_matrix(fn, "a", a, N, columns, lda, 1)) return st;
    if (fp8bs_status st = check_matrix(fn, "b", b, K, columns, ldb, 1)) return st;
    // Offsets inside a tile are 32-bit: 256 rows of codes.
    if (lda > kWide || ldb > kWide) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch above 2^22", fn);
    if (!a_scale || !b_scale) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (scales)", fn);
    if (!aligned4(a_scale) || !aligned4(b_scale)) return fail(FP8BS_ERR_ALIGNMENT, "%s: scales must be 4-byte aligned", fn);
  }
  if (fp8bs_status st = check_apart(fn, {{"y", line(y, G * N * K * elem_size(y_dtype)), false}},
                                    {{"a", matrix_block(a, N, columns, lda, 1), false},
                                     {"b", matrix_block(b, K, columns, ldb, 1), false},
                                     {"a_scale", line(a_scale, N * (columns / 128) * 4), false},
                                     {"b_scale", line(b_scale, K * (columns / 128) * 4), false},
                                     {"padded", line(padded, (G + int64_t(1)) * 4), false}}))
    return st;
  Args args{};
  args.a = a, args.b = b, args.a_scale = a_scale, args.b_scale = b_scale, args.padded = padded, args.y = y;
  args.lda = lda, args.ldb = ldb;
  args.N = static_cast<int32_t>(N), args.K = static_cast<int32_t>(K), args.blocks = static_cast<int32_t>(columns / 128), args.G = G;
  args.accumulate = accumulate;
  // Tiles of 256 x 256, one a CU, where they come in more than four rounds of
  // workgroups or in two to four nearly full ones; of 128 x 128, two a CU, where
  // they nearly fill one.  Measured, float32, us, tiles of 256 / 128 / 64, experts of
  // one depth and of depths that differ by a factor of about four:
  //   mean depth of an expert                       1024: even     uneven      4096: even      uneven
  //   48 experts 1024 x 2048 (1536 tiles of 256)    232 / 265      234 / 252   702 / 762       720 / 771
  //   16 of them (512)                              76 / 78        93 / 94     234 / 257       254 / 267
  //   12 of them (384; 1536 of 128)                 66 / 59        77 / 75     201 / 196       198 / 208
  //   8 of them (256)                               39 / 41        40 / 42     118 / 133       158 / 132
  //   7 experts 1024 x 1024 (448 of 128)            - / 21 / 23    - / 30 / 26 - / 65 / 72     - / 69 / 75
  //   6 of them (384)                               - / 19 / 21    - / 21 / 21 - / 58 / 63     - / 85 / 65
  //   4 of them (256)                               - / 14 / 14    - / 19 / 15 - / 40 / 43     - / 78 / 51
  // Steps of whole blocks have half the barriers and twice the loads under way: 64
  // experts of 512 x 512, 1536 deep, 68 and with half blocks 81; 12 of them in tiles
  // of 64, 4096 deep, 36 and 43.  Where experts have no more than a block or two each,
  // the output is nearly all the work, and half steps let more workgroups share a CU:
  // 16 experts of 1024 x 2048, 256 deep, 40 and 38; 32 of 512 x 1040, 128 deep, in
  // tiles of 64 20 and 18.  More of them help there too: at one block 16 experts of
  // 4096 x 7168 take 365 / 338 / 372, 16 of 1024 x 1024 (1024 of 128) - / 18 / 16.
  // All of that with operands as wide as the experts' tiles.  fp8_quant_grouped_t's
  // have its bound's width, nearly a block an expert more, and experts of one or two
  // blocks count as deeper there: 16 experts of 4096 x 7168 take 371 us so and 336
  // trimmed at one block, 452 and 436 at two, 16 of 1024 x 1024 21 and 18 at two;
  // deeper ones the same.
  const auto tiles = [&](int64_t size) { return G * ((N + size - 1) / size) * ((K + size - 1) / size); };
  const bool bf16 = y_dtype == FP8BS_BF16;
  const int64_t large = tiles(256), rounds = (large + 255) / 256;
  const int64_t blocks = columns / 128;
  if ((rounds > 4 || (large >= 512 && large * 8 >= rounds * 256 * 7)) && blocks > G) return launch<Large>(args, bf16, stream);
  if (blocks <= 2 * G) return tiles(128) >= 1536 ? launch<Half128>(args, bf16, stream) : launch<Half64>(args, bf16, stream);
  return tiles(128) >= 448 ? launch<Whole128>(args, bf16, stream) : launch<Whole64>(args, bf16, stream);
}

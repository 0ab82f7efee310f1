// Attention of new tokens over the paged 8-bit cache, for gfx950.
//
// z = softmax_scale * q . k over the visible positions, out = softmax(z) . v,
// lse = log sum exp z, in one pass over the cache with a running maximum and
// sum per row.  Rows are (token, query head) pairs that share a kv head, so
// that one read of the cache serves all of them.
//
// Both products run on the bf16 matrix instructions, transposed: S^T = K Q^T
// and O^T = V^T P^T.  A lane then owns one row of the softmax (the column of
// the result), and the result of the first product is already laid out as
// the right operand of the second: with 16x16x32 tiles, lane (n, g) holds
// scores of keys 4g .. 4g+3 of two 16-key tiles for row n, and the second
// product may take its 32 keys in any order as long as V^T has the same one.
// Codes are widened to bf16 by an instruction that also multiplies by a power
// of two, so that a page's scale costs nothing and is exact.
//
// Rounding.  Scores, maxima, sums and outputs are float32 until the end.  The
// weights alone are rounded to bf16 (half a step, 2^-8) before the second
// product: a matrix instruction's operands are of one type, V with scales from
// 2^-32 to 2^120 needs bf16's range (float16 ends at 65504), and products of
// float32 run at a sixteenth of the rate.  The sum of weights is of the
// unrounded ones.  The results' error against 64 bits is 2.2e-3 of their norm
// for prompts and 1.7e-3 to 1.8e-3 for single tokens, where the output's own
// rounding to bf16 makes 1.7e-3.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kv_common.hpp"
#include "kv_tiles.hpp"

namespace fp8bs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;

struct AttendParams {
  KvView kv;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part_o;        // [splits, rows of q, head_dim]: unnormalised sums of a split
  float* part_ml;       // [splits, rows of q, 2]: its maximum and sum of weights
  int64_t ld_q, hs_q;
  float scale_log2;     // |softmax_scale| log2 e (a negative scale negates q)
  bool negate;
  int32_t q_heads;
  int32_t window;
  int32_t splits;
  int32_t split_len;    // keys of a split
  FastDiv by_group;     // query heads of one kv head
  FastDiv by_heads;     // kv heads
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
__device__ __forceinline__ bf2 widen_lo(uint32_t w, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false); }
__device__ __forceinline__ bf2 widen_hi(uint32_t w, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true); }
__device__ __forceinline__ bf8 join(bf2 a, bf2 b, bf2 c, bf2 d) { return bf8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y}; }

// Bit 7 of every byte that holds an E4M3 NaN (S.1111.111).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }   // results below 2^-126 become 0
__device__ __forceinline__ bf8 negated(bf8 x) { return __builtin_bit_cast(bf8, __builtin_bit_cast(u32x4, x) ^ 0x80008000u); }

// The rows of one workgroup: rows [r0, r0 + count) of a sequence's n * group
// rows (row = token * group + head within the group) and the keys they see.
struct RowRange {
  Seq s;
  int h;               // kv head
  int last_row;
  int pos_lo, pos_hi;  // positions of the first and the last row
  int key_lo, key_hi;  // keys of this workgroup's split
  const int32_t* table;
};
__device__ __forceinline__ bool find_rows(const AttendParams& p, int b, int h, int64_t r0, int count, int split, int key_align, RowRange& r) {
  const KvView& c = p.kv;
  r.h = h;
  r.s = load_seq(c, b);
  const int64_t rows = int64_t(r.s.n) * p.by_group.d;
  if (r0 >= rows) return false;
  r.last_row = static_cast<int>(min(r0 + count, rows) - 1);
  r.pos_lo = r.s.start + static_cast<int>(p.by_group.div(static_cast<int>(r0)));
  r.pos_hi = r.s.start + static_cast<int>(p.by_group.div(r.last_row));
  const int end = min(r.pos_hi + 1, r.s.end);
  r.key_lo = (p.window > 0 ? max(0, r.pos_lo - p.window + 1) & -key_align : 0) + split * p.split_len;
  r.key_hi = split + 1 == p.splits ? end : min(end, r.key_lo + p.split_len);
  r.table = c.table + b * c.ld_table;
  return true;
}

// One row's result: normalised into out and lse, or as it is into the
// workspace where the keys were split.  `top` is the reference that the
// weights were taken against, in log2 units.
template <int kRun>
__device__ __forceinline__ void put_row(const AttendParams& p, int split, int64_t at, int dim, int head_dim, const f32x4 (&acc)[kRun],
                                        float top, float sum, bool with_lse) {
  if (p.splits > 1) {
    const int64_t prow = int64_t(split) * p.kv.tokens * p.q_heads + at;
#pragma unroll
    for (int i = 0; i < kRun; ++i) *reinterpret_cast<f32x4*>(p.part_o + prow * head_dim + dim + 4 * i) = acc[i];
    if (with_lse) {
      p.part_ml[2 * prow] = top;
      p.part_ml[2 * prow + 1] = sum;
    }
    return;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // a NaN sum stays a NaN
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    *reinterpret_cast<u32x2*>(p.out + at * head_dim + dim + 4 * i) =
        u32x2{pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv)};
  if (p.lse && with_lse) p.lse[at] = ((top == kNegInf ? 0.0f : top) + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------------
// Few rows (a decode step, short prompts): workgroup (b * heads + h, tile of 16
// rows, split) of one kv head over one split of their keys.  The waves take 32-key
// steps in turn and join at the end.  Bound by reading the cache: the codes
// go from memory to registers to the matrix instructions, the next step's
// are in flight while one is computed, and the page numbers and scales of 32
// steps ahead are fetched by the lanes at once.  64 sequences of up to 8192
// tokens with 8 kv heads of 128 take 135 us, 4.9 TB/s of cache.
template <int kD>
struct Step32 {                      // one 32-key step's codes as loaded
  u32x4 k[2][kD / 64];
  uint32_t v[8][kD / 64];
};

template <int kD, int kWaves>
__global__ __launch_bounds__(kWaves * 64, kWaves == 4 ? 3 : 2) void attend_rows_kernel(AttendParams p) {
  constexpr int kU = kD / 64;       // 16-byte loads of a key's dims per lane
  constexpr int kI = kD / 16;       // dims of V per lane: one product each
  constexpr int kStride = 32 * kWaves;
  __shared__ __align__(16) float sh_o[kWaves][16][kD + 4];
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
  const KvView& c = p.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int group = p.by_group.d;
  const int64_t r0 = int64_t(blockIdx.y) * 16;
  RowRange rr;
  const int b = p.by_heads.div(blockIdx.x), split = blockIdx.z;
  if (!find_rows(p, b, blockIdx.x - b * c.heads, r0, 16, split, 32, rr)) return;
  const Seq& s = rr.s;
  const int row = min(static_cast<int>(r0) + n, rr.last_row);
  const int token = p.by_group.div(row);
  const int head = rr.h * group + (row - token * group);
  const int pos = s.start + token;
  const int window = p.window > 0 ? p.window : 0x40000000;   // positions stay below 2^30

  bf8 q[2 * kU];
  {
    const uint16_t* src = p.q + int64_t(s.row0 + token) * p.ld_q + head * p.hs_q + 16 * g;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      q[2 * u] = *reinterpret_cast<const bf8*>(src + 64 * u);
      q[2 * u + 1] = *reinterpret_cast<const bf8*>(src + 64 * u + 8);
    }
    if (p.negate) {
#pragma unroll
      for (int u = 0; u < 2 * kU; ++u) q[u] = negated(q[u]);
    }
  }

  f32x4 o[kI] = {};
  float m = kNegInf, l = 0.0f;
  const int k_off = n * kD + 16 * g, v_off = 4 * g * kD + kI * n;
  const int page_mask = (1 << c.page_shift) - 1;

  for (int run = rr.key_lo + 32 * wave; run < rr.key_hi; run += 32 * kStride) {
    // lane i: page and scales of tile i & 1 of step i >> 1 of this run
    const int my_key = run + (lane >> 1) * kStride + 16 * (lane & 1);
    int my_page = -1;
    if (my_key < rr.key_hi) my_page = rr.table[my_key >> c.page_shift];
    if (my_page >= c.pages) my_page = -1;
    float my_ks = 1.0f, my_vs = 1.0f;
    if (my_page >= 0) {
      my_ks = c.k_scale[int64_t(my_page) * c.heads + rr.h];
      my_vs = c.v_scale[int64_t(my_page) * c.heads + rr.h];
    }
    const int steps = min(32, (rr.key_hi - run + kStride - 1) / kStride);

    auto fetch = [&](int step, Step32<kD>& f) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int page = __builtin_amdgcn_readlane(my_page, 2 * step + t);
        const int key0 = run + step * kStride + 16 * t;
        const int64_t at = (((int64_t(max(page, 0)) * c.heads + rr.h) << c.page_shift) + (key0 & page_mask)) * kD;
        if (page >= 0) {
          const uint8_t* ks = c.k + at;
          const uint8_t* vs = c.v + at;
#pragma unroll
          for (int u = 0; u < kU; ++u) f.k[t][u] = *reinterpret_cast<const u32x4*>(ks + (k_off + 64 * u));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (kU == 2) {
              const u32x2 w = *reinterpret_cast<const u32x2*>(vs + (v_off + j * kD));
              f.v[4 * t + j][0] = w.x;
              f.v[4 * t + j][kU - 1] = w.y;
            } else {
              f.v[4 * t + j][0] = *reinterpret_cast<const uint32_t*>(vs + (v_off + j * kD));
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            f.k[t][u] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[4 * t + j][u] = 0;
          }
        }
      }
    };

    Step32<kD> cur, next;
    fetch(0, cur);
    for (int step = 0; step < steps; ++step) {
      if (step + 1 < steps) fetch(step + 1, next);
      const int kb = run + step * kStride;
      const int page0 = __builtin_amdgcn_readlane(my_page, 2 * step), page1 = __builtin_amdgcn_readlane(my_page, 2 * step + 1);
      const float ks[2] = {__int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_ks), 2 * step)),
                           __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_ks), 2 * step + 1))};
      const float vs[2] = {__int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_vs), 2 * step)),
                           __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_vs), 2 * step + 1))};
      f32x4 z[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 acc = {};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const u32x4 w = cur.k[t][u];
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              join(widen_lo(w.x, ks[t]), widen_hi(w.x, ks[t]), widen_lo(w.y, ks[t]), widen_hi(w.y, ks[t])), q[2 * u], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              join(widen_lo(w.z, ks[t]), widen_hi(w.z, ks[t]), widen_lo(w.w, ks[t]), widen_hi(w.w, ks[t])), q[2 * u + 1], acc, 0, 0, 0);
        }
        z[t] = acc;
      }
      // a step that some row does not see in whole
      const bool edge = kb + 31 >= rr.key_hi || kb + 31 > rr.pos_lo || rr.pos_hi - kb >= window || page0 < 0 || page1 < 0;
      if (edge) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kb + 16 * t + 4 * g + r;
            const bool see = (t ? page1 : page0) >= 0 && key < rr.key_hi && key <= pos && pos - key < window;
            z[t][r] = see ? z[t][r] : kNegInf;
          }
        }
      }
      float top = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])), fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__ballot(top > m)) {
        const float m_new = fmaxf(m, top);
        const float alpha = m == m_new ? 1.0f : exp2_fast((m - m_new) * p.scale_log2);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < kI; ++i) o[i] *= alpha;
      }
      const float base = m == kNegInf ? 0.0f : m * p.scale_log2;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = exp2_fast(__builtin_fmaf(z[j >> 2][j & 3], p.scale_log2, -base));
      l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
      if (edge) {
        // a NaN value reaches only the rows that see its key: the product
        // would also carry it into rows whose weight is 0
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int u = 0; u < kU; ++u) bad |= nan_bytes(cur.v[j][u]);
        }
        if (__ballot(bad != 0)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t hit = 0;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              const uint32_t nb = nan_bytes(cur.v[j][u]);
              hit |= nb;
              cur.v[j][u] &= ~((nb >> 7) * 0xffu);
            }
            const uint64_t who = __ballot(hit != 0);
            if (((who >> (16 * g)) & 0xffffu) && z[j >> 2][j & 3] != kNegInf) l = __builtin_nanf("");
          }
        }
      }
      // weights as bf16: see the head of the file
      const bf8 pb = __builtin_bit_cast(bf8, u32x4{pack2(w[0], w[1]), pack2(w[2], w[3]), pack2(w[4], w[5]), pack2(w[6], w[7])});
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint32_t lo[4], hi[4];      // byte pairs (key 2j, key 2j + 1) of two dims each
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = __builtin_amdgcn_perm(cur.v[2 * j + 1][u], cur.v[2 * j][u], 0x05010400u);
          hi[j] = __builtin_amdgcn_perm(cur.v[2 * j + 1][u], cur.v[2 * j][u], 0x07030602u);
        }
        o[4 * u + 0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            join(widen_lo(lo[0], vs[0]), widen_lo(lo[1], vs[0]), widen_lo(lo[2], vs[1]), widen_lo(lo[3], vs[1])), pb, o[4 * u + 0], 0, 0, 0);
        o[4 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            join(widen_hi(lo[0], vs[0]), widen_hi(lo[1], vs[0]), widen_hi(lo[2], vs[1]), widen_hi(lo[3], vs[1])), pb, o[4 * u + 1], 0, 0, 0);
        o[4 * u + 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            join(widen_lo(hi[0], vs[0]), widen_lo(hi[1], vs[0]), widen_lo(hi[2], vs[1]), widen_lo(hi[3], vs[1])), pb, o[4 * u + 2], 0, 0, 0);
        o[4 * u + 3] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            join(widen_hi(hi[0], vs[0]), widen_hi(hi[1], vs[0]), widen_hi(hi[2], vs[1]), widen_hi(hi[3], vs[1])), pb, o[4 * u + 3], 0, 0, 0);
      }
      cur = next;
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // join the waves
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int i = 0; i < kI; i += 4)
      *reinterpret_cast<f32x4*>(&sh_o[wave][n][kI * (4 * g + r) + i]) = f32x4{o[i][r], o[i + 1][r], o[i + 2][r], o[i + 3][r]};
  }
  if (g == 0) {
    sh_m[wave][n] = m == kNegInf ? kNegInf : m * p.scale_log2;
    sh_l[wave][n] = l;
  }
  __syncthreads();
  const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;   // row and run of kI dims
  if (jr >= 16) return;
  const int jrow = static_cast<int>(r0) + jr;
  if (jrow > rr.last_row) return;
  const int jt = p.by_group.div(jrow);
  float top = kNegInf;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sh_m[w][jr]);
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
  f32x4 acc[kI / 4] = {};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = exp2_fast(sh_m[w][jr] - base);
    sum += f * sh_l[w][jr];
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) acc[i] += f * *reinterpret_cast<const f32x4*>(&sh_o[w][jr][kI * jc + 4 * i]);
  }
  // a NaN in any dim is the row's
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kI; ++i) bad |= acc[i >> 2][i & 3] != acc[i >> 2][i & 3];
  if ((__ballot(bad) >> (threadIdx.x & 48)) & 0xffffu) sum = __builtin_nanf("");
  const int64_t at = int64_t(s.row0 + jt) * p.q_heads + rr.h * group + (jrow - jt * group);
  put_row<kI / 4>(p, split, at, kI * jc, kD, acc, top, sum, jc == 0);
}

// ---------------------------------------------------------------------------
// Many rows (prompts, chunks of prompts): workgroup (tile of 128 rows, kv
// head; split), 32 rows a wave, over 64-key tiles.  A wave issues a vector
// instruction every 8 cycles at best, so the two waves a SIMD that these
// registers allow spend a tile's time on, in this order, the softmax, the
// matrix instructions and the widening, and overlap only each other: prompts
// of 8192 tokens and of 2179 over 6522, 32 heads of 128, take 788 us, 0.94
// PFLOP/s (256-row tiles, one wave a SIMD, took 1390 us).  The four waves
// widen a tile's codes once for all of them, into LDS as bf16: K as
// [key][dim], V transposed as [dim][key], keys in the order in which the
// first product leaves the weights (16-key runs, slot 8 h + j = key 4 h + j
// or, from j = 4, 8 + 4 h + j - 4).  Wave w loads and widens keys 16 w ..
// 16 w + 15, which lie in one page.  32x32x16 products: lane (i, h) = (lane & 31, lane >> 5) owns
// row i; register r of S^T is key 8 (r / 4) + 4 h + r % 4.
// 16-byte chunks of an LDS row are swizzled so that both the widening's
// writes and the products' reads spread over the 64 banks: 16 lanes of a read
// hit 16 different chunks of 256 bytes.
constexpr float kSlack = 8.0f;     // log2 units by which a row's maximum may outgrow its reference

// A wave on the GPU, for find_tile: lane i holds sequence i's place.
struct LaneWave {
  int lane;
  TilePlace first;
  template <class F>
  __device__ __forceinline__ int sum(F f) const {
    int v = f(lane, first);
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return __builtin_amdgcn_readfirstlane(v);
  }
  template <class F>
  __device__ __forceinline__ uint64_t ballot(F f) const { return __ballot(f(lane, first)); }
};

// max over lanes l and l ^ 32
__device__ __forceinline__ float halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <int kD>
struct __align__(16) Tiles {
  uint16_t k[64][kD];
  uint16_t v[kD][64];
  uint32_t nans[4];      // keys of the run whose value holds a NaN (edge tiles only)
};
template <int kD> __device__ __forceinline__ int k_chunk(int key, int chunk) { return (chunk ^ (kD == 128 ? key & 15 : ((key >> 2) ^ (key << 1)) & 7)) * 8; }
__device__ __forceinline__ int v_chunk(int dim, int chunk) { return (chunk ^ (((dim >> 2) ^ (dim << 1)) & 7)) * 8; }

template <int kD>
__global__ __launch_bounds__(256, 2) void attend_tiles_kernel(AttendParams p) {
  constexpr int kC = kD / 16;        // 16-dim steps of the first product
  constexpr int kT = kD / 32;        // 32-dim tiles of the second
  constexpr int kRows = 128;
  __shared__ Tiles<kD> sh[2];
  const KvView& c = p.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i32 = lane & 31, h32 = lane >> 5;
  const int group = p.by_group.d;
  int b, tile_y;
  const int h = blockIdx.x % c.heads, split = blockIdx.z;
  if (!find_tile(LaneWave{lane, tile_place(c, lane, group)}, c, blockIdx.x / c.heads, group, b, tile_y)) return;
  const int64_t r0 = int64_t(tile_y) * kRows;
  RowRange rr;
  if (!find_rows(p, b, h, r0, kRows, split, 64, rr)) return;
  const Seq& s = rr.s;
  const int window = p.window > 0 ? p.window : 0x40000000;

  const int w0 = static_cast<int>(r0) + wave * 32;
  const bool has_rows = w0 <= rr.last_row;
  int wave_lo = 0, wave_hi = -1;     // positions of the wave's rows
  if (has_rows) {
    wave_lo = s.start + static_cast<int>(p.by_group.div(w0));
    wave_hi = s.start + static_cast<int>(p.by_group.div(min(w0 + 31, rr.last_row)));
  }
  const int row = min(w0 + i32, rr.last_row);
  const int token = p.by_group.div(row);
  const int head = rr.h * group + (row - token * group);
  const int pos = s.start + token;
  bf8 q[kC];
  {
    const uint16_t* src = p.q + int64_t(s.row0 + token) * p.ld_q + head * p.hs_q + 8 * h32;
#pragma unroll
    for (int u = 0; u < kC; ++u) {
      q[u] = *reinterpret_cast<const bf8*>(src + 16 * u);
      if (p.negate) q[u] = negated(q[u]);
    }
  }

  const int page_mask = (1 << c.page_shift) - 1;
  // V: lane (group of 8 slots h32, dims kD / 32 * i32 ..)
  constexpr int kVB = kD / 32;       // bytes of V a lane takes of each of its 8 keys
  uint32_t raw_k[kD / 16], raw_v[8];
  // Lane i: page and scales of this wave's run of tile first_tile + i, and
  // which runs of that tile have no page.  One look serves 62 tiles.
  int first_tile = 0, my_page = -1, my_unseen = 0;
  float my_ks = 1.0f, my_vs = 1.0f;
  auto find_pages = [&](int tile) {
    first_tile = tile;
    my_unseen = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key0 = rr.key_lo + 64 * (tile + lane) + 16 * r;
      const int page = key0 < rr.key_hi ? rr.table[key0 >> c.page_shift] : -1;
      const bool none = page < 0 || page >= c.pages;
      if (none) my_unseen |= 1 << r;
      if (r == wave) my_page = none ? -1 : page;
    }
    if (my_page >= 0) {
      my_ks = c.k_scale[int64_t(my_page) * c.heads + rr.h];
      my_vs = c.v_scale[int64_t(my_page) * c.heads + rr.h];
    }
  };
  auto of_tile = [&](float x, int tile) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), tile - first_tile)); };
  auto load = [&](int tile) {
    const int page = __builtin_amdgcn_readlane(my_page, tile - first_tile);
    if (page >= 0) {
      const int64_t base = (((int64_t(page) * c.heads + rr.h) << c.page_shift) + ((rr.key_lo + 64 * tile + 16 * wave) & page_mask)) * kD;
      const uint8_t* kp = c.k + base + ((lane >> 2) * kD + (lane & 3) * 16);
#pragma unroll
      for (int u = 0; u < kD / 64; ++u) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(kp + 64 * u);
        raw_k[4 * u] = x.x; raw_k[4 * u + 1] = x.y; raw_k[4 * u + 2] = x.z; raw_k[4 * u + 3] = x.w;
      }
      const uint8_t* vp = c.v + base + (4 * h32 * kD + kVB * i32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* src = vp + ((j & 3) + 8 * (j >> 2)) * kD;
        if constexpr (kVB == 4) raw_v[j] = *reinterpret_cast<const uint32_t*>(src);
        else raw_v[j] = *reinterpret_cast<const uint16_t*>(src);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kD / 16; ++u) raw_k[u] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) raw_v[j] = 0;
    }
  };
  // a tile that some row of the workgroup does not see in whole
  auto is_edge = [&](int kb) { return kb + 63 >= rr.key_hi || kb + 63 > rr.pos_lo || rr.pos_hi - kb >= window; };
  auto store = [&](int tile, Tiles<kD>& t) {
    const float ks = of_tile(my_ks, tile), vs = of_tile(my_vs, tile);
    if (is_edge(rr.key_lo + 64 * tile)) {
      uint32_t nans = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t nb = nan_bytes(raw_v[j]);
        raw_v[j] &= ~((nb >> 7) * 0xffu);
        const uint64_t who = __ballot(nb != 0);
        const int k4 = (j & 3) + 8 * (j >> 2);
        if (who & 0xffffffffu) nans |= 1u << k4;
        if (who >> 32) nans |= 1u << (k4 + 4);
      }
      if (lane == 0) t.nans[wave] = nans;
    }
    const int key = 16 * wave + (lane >> 2);
#pragma unroll
    for (int u = 0; u < kD / 32; ++u) {
      const bf8 x = join(widen_lo(raw_k[2 * u], ks), widen_hi(raw_k[2 * u], ks), widen_lo(raw_k[2 * u + 1], ks), widen_hi(raw_k[2 * u + 1], ks));
      *reinterpret_cast<bf8*>(&t.k[key][k_chunk<kD>(key, (u >> 1) * 8 + (lane & 3) * 2 + (u & 1))]) = x;
    }
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = __builtin_amdgcn_perm(raw_v[2 * j + 1], raw_v[2 * j], 0x05010400u);
      if constexpr (kVB == 4) hi[j] = __builtin_amdgcn_perm(raw_v[2 * j + 1], raw_v[2 * j], 0x07030602u);
    }
    const int dim = kVB * i32, chunk = 2 * wave + h32;
    auto put = [&](int d, bf8 x) { *reinterpret_cast<bf8*>(&t.v[dim + d][v_chunk(dim + d, chunk)]) = x; };
    put(0, join(widen_lo(lo[0], vs), widen_lo(lo[1], vs), widen_lo(lo[2], vs), widen_lo(lo[3], vs)));
    put(1, join(widen_hi(lo[0], vs), widen_hi(lo[1], vs), widen_hi(lo[2], vs), widen_hi(lo[3], vs)));
    if constexpr (kVB == 4) {
      put(2, join(widen_lo(hi[0], vs), widen_lo(hi[1], vs), widen_lo(hi[2], vs), widen_lo(hi[3], vs)));
      put(3, join(widen_hi(hi[0], vs), widen_hi(hi[1], vs), widen_hi(hi[2], vs), widen_hi(hi[3], vs)));
    }
  };

  v16f o[kT] = {};
  float m = kNegInf, l = 0.0f;

  if (rr.key_lo < rr.key_hi) {
    find_pages(0);
    load(0);
    store(0, sh[0]);
    load(1);
  }
  __syncthreads();
  for (int n = 0, kb = rr.key_lo; kb < rr.key_hi; ++n, kb += 64) {
    const Tiles<kD>& tile = sh[n & 1];
    if (n + 2 - first_tile >= 64) find_pages(n);
    if (kb + 64 < rr.key_hi) {
      store(n + 1, sh[~n & 1]);
      load(n + 2);
    }
    if (has_rows && kb <= wave_hi && (p.window == 0 || kb + 63 > wave_lo - window)) {
      v16f z[2] = {};
#pragma unroll
      for (int u = 0; u < kC; ++u) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const int key = 32 * kt + i32;
          const bf8 a = *reinterpret_cast<const bf8*>(&tile.k[key][k_chunk<kD>(key, 2 * u + h32)]);
          z[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[u], z[kt], 0, 0, 0);
        }
      }
      const int unseen = __builtin_amdgcn_readlane(my_unseen, n - first_tile);
      if (unseen || kb + 63 >= rr.key_hi || kb + 63 > wave_lo || wave_hi - kb >= window) {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          const int key = kb + 32 * (r >> 4) + 8 * ((r & 15) >> 2) + 4 * h32 + (r & 3);
          const bool see = key < rr.key_hi && key <= pos && pos - key < window && !(unseen >> (r >> 3) & 1);
          z[r >> 4][r & 15] = see ? z[r >> 4][r & 15] : kNegInf;
        }
      }
      float top = fmaxf(z[0][0], z[0][1]);
#pragma unroll
      for (int r = 2; r < 32; r += 2) top = fmaxf(fmaxf(top, z[r >> 4][r & 15]), z[r >> 4][(r & 15) + 1]);
      top = halves_max(top);
      // the reference moves only when the maximum has outgrown it: weights
      // stay below 2^kSlack, and the accumulators are rarely rescaled
      if (__ballot((top - m) * p.scale_log2 > kSlack || (m == kNegInf && top > kNegInf))) {
        const float m_new = fmaxf(m, top);
        const float alpha = m == m_new ? 1.0f : exp2_fast((m - m_new) * p.scale_log2);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kT; ++d) o[d] *= alpha;
      }
      const float base = m == kNegInf ? 0.0f : m * p.scale_log2;
      if (is_edge(kb)) {
        const uint32_t n01 = tile.nans[0] | tile.nans[1] << 16, n23 = tile.nans[2] | tile.nans[3] << 16;
        if (__builtin_amdgcn_readfirstlane(n01 | n23)) {
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            const int key = 8 * ((r & 15) >> 2) + 4 * h32 + (r & 3);
            if (((r < 16 ? n01 : n23) >> key & 1) && z[r >> 4][r & 15] != kNegInf) l = __builtin_nanf("");
          }
        }
      }
      float part[4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          e[r] = exp2_fast(__builtin_fmaf(z[k >> 1][8 * (k & 1) + r], p.scale_log2, -base));
          part[r & 3] += e[r];
        }
        // weights as bf16: see the head of the file
        const bf8 w = __builtin_bit_cast(bf8, u32x4{pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7])});
#pragma unroll
        for (int d = 0; d < kT; ++d) {
          const int dim = 32 * d + i32;
          const bf8 a = *reinterpret_cast<const bf8*>(&tile.v[dim][v_chunk(dim, 2 * k + h32)]);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, w, o[d], 0, 0, 0);
        }
      }
      l += (part[0] + part[1]) + (part[2] + part[3]);
    }
    __syncthreads();
  }

  if (!has_rows) return;
  // a NaN in any dim is the row's
  bool bad = false;
#pragma unroll
  for (int d = 0; d < kT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= o[d][r] != o[d][r];
  }
  if (bad) l = __builtin_nanf("");
  const float sum = l + __shfl_xor(l, 32);
  const float top = m == kNegInf ? kNegInf : m * p.scale_log2;
  if (w0 + i32 > rr.last_row) return;
  const int64_t at = int64_t(s.row0 + token) * p.q_heads + head;
#pragma unroll
  for (int d = 0; d < kT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const f32x4 x[1] = {{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]}};
      put_row<1>(p, split, at, 32 * d + 2 * r + 4 * h32, kD, x, top, sum, d == 0 && r == 0 && h32 == 0);
    }
  }
}

// ---------------------------------------------------------------------------
// Joins many splits: workgroup (row of a sequence, b).  16 lanes cover a row's
// dims, the 16 such groups of the workgroup take the splits in turn.
constexpr int kMaxSplits = 512;
template <int kD>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int kI = kD / 16;
  __shared__ float sh_w[kMaxSplits];
  __shared__ __align__(16) float sh_o[16][kD + 4];
  __shared__ float red[8];
  const KvView& c = p.kv;
  const Seq s = load_seq(c, blockIdx.y);
  const int64_t r = blockIdx.x;
  if (r >= int64_t(s.n) * p.q_heads) return;
  const int64_t at = int64_t(s.row0) * p.q_heads + r;
  const int64_t pitch = int64_t(c.tokens) * p.q_heads;
  const int tid = threadIdx.x;
  float mine[2], sums[2], top = kNegInf;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = tid + 256 * i;
    mine[i] = kNegInf;
    sums[i] = 0.0f;
    if (k < p.splits) {
      mine[i] = p.part_ml[2 * (k * pitch + at)];
      sums[i] = p.part_ml[2 * (k * pitch + at) + 1];
    }
    top = fmaxf(top, mine[i]);
  }
  top = wave_max(top);
  if ((tid & 63) == 0) red[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = tid + 256 * i;
    const float f = exp2_fast(mine[i] - base);
    if (k < p.splits) sh_w[k] = f;
    sum += f * sums[i];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) red[4 + (tid >> 6)] = sum;
  __syncthreads();
  sum = (red[4] + red[5]) + (red[6] + red[7]);
  const int jc = tid & 15, jg = tid >> 4;
  f32x4 acc[kI / 4] = {};
  for (int k = jg; k < p.splits; k += 16) {
    const float f = sh_w[k];
    if (f == 0.0f) continue;                    // a split that saw nothing, or nothing that counts
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) acc[i] += f * *reinterpret_cast<const f32x4*>(p.part_o + (k * pitch + at) * kD + kI * jc + 4 * i);
  }
#pragma unroll
  for (int i = 0; i < kI / 4; ++i) *reinterpret_cast<f32x4*>(&sh_o[jg][kI * jc + 4 * i]) = acc[i];
  __syncthreads();
  if (tid < kD) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) x += sh_o[k][tid];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    reinterpret_cast<__bf16*>(p.out)[at * kD + tid] = static_cast<__bf16>(x * inv);
    if (p.lse && tid == 0) p.lse[at] = (base + log2f(sum)) * kLn2;
  }
}

// Joins at most kFewSplits splits (chunks of prompts have many rows): 16 lanes
// take a whole row, 16 rows a workgroup (49000 rows of 64 in two splits: the
// call takes 88 us, and 130 us with a workgroup a row).
constexpr int kFewSplits = 8;
template <int kD>
__global__ __launch_bounds__(256) void attend_join_few_kernel(AttendParams p) {
  constexpr int kI = kD / 16;
  const KvView& c = p.kv;
  const Seq s = load_seq(c, blockIdx.y);
  const int64_t r = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (r >= int64_t(s.n) * p.q_heads) return;
  const int64_t at = int64_t(s.row0) * p.q_heads + r, pitch = int64_t(c.tokens) * p.q_heads;
  const int jc = threadIdx.x & 15;
  float m[kFewSplits], l[kFewSplits], top = kNegInf;
#pragma unroll
  for (int k = 0; k < kFewSplits; ++k) {
    m[k] = kNegInf;
    l[k] = 0.0f;
    if (k < p.splits) {
      m[k] = p.part_ml[2 * (k * pitch + at)];
      l[k] = p.part_ml[2 * (k * pitch + at) + 1];
    }
    top = fmaxf(top, m[k]);
  }
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
  f32x4 acc[kI / 4] = {};
#pragma unroll
  for (int k = 0; k < kFewSplits; ++k) {
    if (k >= p.splits) break;
    const float f = exp2_fast(m[k] - base);
    sum += f * l[k];
    if (f == 0.0f) continue;
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) acc[i] += f * *reinterpret_cast<const f32x4*>(p.part_o + (k * pitch + at) * kD + kI * jc + 4 * i);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < kI / 4; ++i)
    *reinterpret_cast<u32x2*>(p.out + at * kD + kI * jc + 4 * i) =
        u32x2{pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv)};
  if (p.lse && jc == 0) p.lse[at] = (base + log2f(sum)) * kLn2;
}

// How a call is cut up, from its sizes alone.
struct Plan {
  int64_t splits, split_len, tile_rows, row_tiles, workspace;
  int waves;
};
Plan make_plan(const KvView& v, int64_t head_dim, int64_t q_heads, int64_t window) {
  Plan plan{};
  const int64_t group = q_heads / v.heads;
  const int64_t rows = int64_t(v.max_new) * group;
  plan.splits = plan.split_len = 1;
  plan.waves = 4;
  if (rows == 0) return plan;
  int64_t span = v.max_len;
  if (window > 0) span = std::min(span, window + (128 + group - 1) / group + 64);
  span = std::max<int64_t>(span, 1);
  // 16-row tiles read the keys once for each of them, but start at once and
  // keep the whole chip busy; 128-row tiles widen a key once for 128 rows.  64
  // sequences over up to 8192 tokens, 8 kv heads: with 32 rows each 177 us in
  // tiles of 16 and 203 in tiles of 128, with 64 rows 271 and 208.  Small
  // calls: 64 tokens over 500, 256 rows, 8.8 and 22.9 us; 512 tokens, 2048
  // rows, 15.7 and 22.7; 1000 tokens, 4000 rows (2 10^6 row tiles times keys),
  // 37.0 and 36.5; two prompts of 300 over 3000, 1200 rows (3.6 10^6), 47.6
  // and 45.2.
  const int64_t few = (rows + 15) / 16;
  const bool narrow = few <= 2 || (few <= 65535 && few * v.batch * v.heads <= (int64_t(3) << 19) / span);
  plan.tile_rows = narrow ? 16 : 128;
  // narrow: of one sequence; else of all, at most
  plan.row_tiles = narrow ? few : int64_t(v.tokens) * group / 128 + v.batch;
  const int64_t units = plan.row_tiles * (narrow ? v.batch : 1) * v.heads;
  // Rows: splits fill the chip once, with 3 workgroups a CU.  More of them
  // only add to the join: 64 sequences of 1024 to 8192 tokens take 136 us
  // unsplit and 145 us in 8 splits, one of 100003 tokens 47.7 us in 87 splits
  // and 49 us in 157.  A split is 128 keys at least, a step of the four waves
  // (one sequence of 6000 tokens: 11.6 us, with 512 at least 13.3).  Tiles:
  // 1024, twice what fits of heads of 128, since tiles are an upper bound
  // (chunks of up to 512 tokens, 392 workgroups: 106 us unsplit, 88 us in two
  // splits, 104 us in three).
  // Known weakness: max_new and max_len are the largest sequence's, and the
  // others get its plan.  64 single tokens, one over 100000 and 63 over 1000,
  // are not split and take 1002 us (66 by their bytes; the long one alone 41);
  // 63 single tokens and one chunk of 512 over 8192 each get tiles of 128 rows
  // and take 403 us (apart 180 + 174).
  const int64_t slots = narrow ? 768 : 1024;
  int64_t want = slots / units;
  want = std::max<int64_t>(1, std::min<int64_t>({want, span / (narrow ? 128 : 512), kMaxSplits}));
  // Short caches: 8 waves of one workgroup join faster than two launches do.
  // One sequence, 8 kv heads of 128: 1025 tokens 10.5 us, split 11.7; 2000
  // tokens 15.8 us, split 11.7.  Heads of 64: 2000 tokens 10.3 and 11.7.  30
  // sequences over 1500 tokens: 15.6 and 17.2.
  if (narrow && units <= 256 && span * head_dim <= (units <= 128 ? 1280 : 2048) * 128) {
    want = 1;
    plan.waves = 8;
  }
  plan.split_len = ((span + want - 1) / want + 127) / 128 * 128;
  plan.splits = (span + plan.split_len - 1) / plan.split_len;
  if (plan.splits > 1) plan.workspace = plan.splits * v.tokens * q_heads * (head_dim + 2) * 4;
  return plan;
}

fp8bs_status check_attention(const char* fn, const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch,
                             const fp8bs_kv_attention_args* a, bool pointers, KvView* view) {
  if (!a) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  if (fp8bs_status st = check_kv(fn, cache, batch, pointers, view)) return st;
  if (a->q_heads < 1 || a->q_heads > 65535 || a->q_heads % cache->kv_heads)
    return fail(FP8BS_ERR_SHAPE, "%s: q_heads %lld is not a multiple of kv_heads %lld", fn, (long long)a->q_heads,
                (long long)cache->kv_heads);
  if (a->window < 0 || a->window > (1 << 30)) return fail(FP8BS_ERR_INVALID_ARG, "%s: window %lld out of range", fn, (long long)a->window);
  if (!std::isfinite(a->softmax_scale)) return fail(FP8BS_ERR_INVALID_ARG, "%s: softmax_scale is not finite", fn);
  if (int64_t(view->max_new) * (a->q_heads / cache->kv_heads) >= (int64_t(1) << 31) || batch->batch * cache->kv_heads >= (int64_t(1) << 31) ||
      !mul_fits(batch->tokens, a->q_heads * cache->head_dim, kMaxBytes / 2))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: more than 2^31 rows of a sequence or more output than any allocation", fn);
  return FP8BS_OK;
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" int64_t fp8_kv_attention_workspace(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch, const fp8bs_kv_attention_args* a) {
  KvView v;
  if (check_attention("fp8_kv_attention_workspace", cache, batch, a, false, &v)) return -1;
  return make_plan(v, cache->head_dim, a->q_heads, a->window).workspace;
}

extern "C" fp8bs_status fp8_kv_attention(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch, const fp8bs_kv_attention_args* a,
                                         hipStream_t stream) {
  const char* fn = "fp8_kv_attention";
  AttendParams p{};
  if (fp8bs_status st = check_attention(fn, cache, batch, a, true, &p.kv)) return st;
  const int64_t d = cache->head_dim, t = batch->tokens;
  if (t == 0) return FP8BS_OK;
  if (fp8bs_status st = check_rows(fn, "q", a->q, t, a->q_heads, d, a->ld_q, a->hs_q)) return st;
  if (fp8bs_status st = check_rows(fn, "out", a->out, t, a->q_heads, d, a->q_heads * d, d)) return st;
  if (!aligned4(a->lse)) return fail(FP8BS_ERR_ALIGNMENT, "%s: lse must be 4-byte aligned", fn);
  const Plan plan = make_plan(p.kv, d, a->q_heads, a->window);
  if (plan.row_tiles * cache->kv_heads >= (int64_t(1) << 23) || batch->batch * cache->kv_heads >= (int64_t(1) << 23))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: 2^23 or more workgroups", fn);
  if (plan.workspace) {
    if (!a->workspace || a->workspace_bytes < plan.workspace)
      return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace of %lld bytes is needed, %lld given", fn, (long long)plan.workspace,
                  (long long)(a->workspace ? a->workspace_bytes : 0));
    if (!aligned16(a->workspace)) return fail(FP8BS_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
  }
  p.q = static_cast<const uint16_t*>(a->q);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = p.part_o ? p.part_o + plan.splits * t * a->q_heads * d : nullptr;
  p.ld_q = a->ld_q;
  p.hs_q = a->hs_q;
  // not 0, which would make masked scores NaN
  p.scale_log2 = std::max(static_cast<float>(std::fabs(a->softmax_scale) * 1.4426950408889634), 1e-36f);
  p.negate = a->softmax_scale < 0;
  p.q_heads = static_cast<int32_t>(a->q_heads);
  p.window = static_cast<int32_t>(a->window);
  p.splits = static_cast<int32_t>(plan.splits);
  p.split_len = static_cast<int32_t>(plan.split_len);
  p.by_group = FastDiv(static_cast<uint32_t>(a->q_heads / cache->kv_heads));
  p.by_heads = FastDiv(static_cast<uint32_t>(cache->kv_heads));
  const uint32_t heads = static_cast<uint32_t>(cache->kv_heads), seqs = static_cast<uint32_t>(batch->batch);
  const uint32_t splits = static_cast<uint32_t>(plan.splits), row_tiles = static_cast<uint32_t>(plan.row_tiles);
  begin_launch();
  if (plan.tile_rows == 16) {
    // splits last: the later ones are empty in short sequences, and would fall
    // on the same shader engines if they were neighbours
    const dim3 grid(seqs * heads, row_tiles, splits);
    if (plan.waves == 4) {
      if (d == 64) hipLaunchKernelGGL((attend_rows_kernel<64, 4>), grid, dim3(256), 0, stream, p);
      else hipLaunchKernelGGL((attend_rows_kernel<128, 4>), grid, dim3(256), 0, stream, p);
    } else {
      if (d == 64) hipLaunchKernelGGL((attend_rows_kernel<64, 8>), grid, dim3(512), 0, stream, p);
      else hipLaunchKernelGGL((attend_rows_kernel<128, 8>), grid, dim3(512), 0, stream, p);
    }
  } else {
    // kv heads fastest: with 8 of them each XCD's L2 holds one head's keys.
    // Then row tiles in falling order: neighbours, which go to different
    // shader engines in turn, have alike amounts of work
    const dim3 grid(heads * row_tiles, 1, splits);
    if (d == 64) hipLaunchKernelGGL(attend_tiles_kernel<64>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(attend_tiles_kernel<128>, grid, dim3(256), 0, stream, p);
  }
  if (plan.splits > 1) {
    const uint32_t jrows = static_cast<uint32_t>(int64_t(p.kv.max_new) * a->q_heads);
    if (plan.splits <= kFewSplits) {
      const dim3 jgrid((jrows + 15) / 16, seqs);
      if (d == 64) hipLaunchKernelGGL(attend_join_few_kernel<64>, jgrid, dim3(256), 0, stream, p);
      else hipLaunchKernelGGL(attend_join_few_kernel<128>, jgrid, dim3(256), 0, stream, p);
    } else {
      const dim3 jgrid(jrows, seqs);
      if (d == 64) hipLaunchKernelGGL(attend_join_kernel<64>, jgrid, dim3(256), 0, stream, p);
      else hipLaunchKernelGGL(attend_join_kernel<128>, jgrid, dim3(256), 0, stream, p);
    }
  }
  return check_launch(fn);
}

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
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kv_common.hpp"

namespace fp8bs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

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
  float scale_log2;     // softmax_scale * log2 e
  int32_t q_heads;
  int32_t window;
  int32_t splits;
  int32_t split_len;    // keys of a split
  FastDiv by_group;     // query heads of one kv head
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
__device__ __forceinline__ bf2 widen_lo(uint32_t w, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false); }
__device__ __forceinline__ bf2 widen_hi(uint32_t w, float s) { return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true); }
__device__ __forceinline__ bf8 join(bf2 a, bf2 b, bf2 c, bf2 d) { return bf8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y}; }

// Bit 7 of every byte that holds an E4M3 NaN (S.1111.111).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Where the keys of one 16-key tile lie: nowhere (seen = false) if the tile
// starts past the end or its page number is not a page.
struct Tile16 {
  bool seen;
  const uint8_t* k;
  const uint8_t* v;
  float ks, vs;
};
template <int kD>
__device__ __forceinline__ Tile16 find_tile(const KvView& c, const int32_t* table, int h, int key0, int end) {
  Tile16 t{false, c.k, c.v, 1.0f, 1.0f};
  if (key0 >= end) return t;
  const int page = __builtin_amdgcn_readfirstlane(table[key0 >> c.page_shift]);
  if (page < 0 || page >= c.pages) return t;
  t.seen = true;
  const int64_t slot = int64_t(page) * c.heads + h;
  const int64_t at = ((slot << c.page_shift) + (key0 & ((1 << c.page_shift) - 1))) * kD;
  t.k += at;
  t.v += at;
  t.ks = c.k_scale[slot];
  t.vs = c.v_scale[slot];
  return t;
}

constexpr int kWaves = 4;

// Workgroup (split, row tile, b * heads + h): 16 rows of one kv head over one
// split of their keys.  The waves take 32-key steps in turn and join at the
// end.
template <int kD>
__global__ __launch_bounds__(kWaves * 64) void attend_rows_kernel(AttendParams p) {
  constexpr int kU = kD / 64;       // 16-byte loads of a key's dims per lane
  constexpr int kI = kD / 16;       // dims of V per lane: one product each
  __shared__ __align__(16) float sh_o[kWaves][16][kD + 4];
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16];
  const KvView& c = p.kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int b = blockIdx.z / c.heads, h = blockIdx.z - b * c.heads;
  const int group = p.by_group.d;
  const Seq s = load_seq(c, b);
  const int64_t rows = int64_t(s.n) * group;
  const int64_t r0 = int64_t(blockIdx.y) * 16;
  if (r0 >= rows) return;
  const int32_t* table = c.table + b * c.ld_table;

  const int last_row = static_cast<int>(min(r0 + 15, rows - 1));
  const int row = min(static_cast<int>(r0) + n, last_row);
  const int token = p.by_group.div(row);
  const int head = h * group + (row - token * group);
  const int pos = s.start + token;
  const int pos_lo = s.start + static_cast<int>(p.by_group.div(static_cast<int>(r0)));
  const int pos_hi = s.start + static_cast<int>(p.by_group.div(last_row));
  int key_lo = p.window > 0 ? max(0, pos_lo - p.window + 1) & ~31 : 0;
  const int key_end = min(pos_hi + 1, s.end);
  key_lo += blockIdx.x * p.split_len;
  const int key_hi = blockIdx.x + 1 == uint32_t(p.splits) ? key_end : min(key_end, key_lo + p.split_len);

  bf8 q[2 * kU];
  {
    const uint16_t* src = p.q + int64_t(s.row0 + token) * p.ld_q + head * p.hs_q + 16 * g;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      q[2 * u] = *reinterpret_cast<const bf8*>(src + 64 * u);
      q[2 * u + 1] = *reinterpret_cast<const bf8*>(src + 64 * u + 8);
    }
  }

  f32x4 o[kI] = {};
  float m = kNegInf, l = 0.0f;
  for (int kb = key_lo + 32 * wave; kb < key_hi; kb += 32 * kWaves) {
    f32x4 z[2];
    uint32_t v[8][kI / 4];
    float vs[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int key0 = kb + 16 * t;
      const Tile16 tile = find_tile<kD>(c, table, h, key0, key_hi);
      vs[t] = tile.vs;
      f32x4 acc = {};
      if (tile.seen) {
        const uint8_t* ksrc = tile.k + n * kD + 16 * g;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(ksrc + 64 * u);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              join(widen_lo(w.x, tile.ks), widen_hi(w.x, tile.ks), widen_lo(w.y, tile.ks), widen_hi(w.y, tile.ks)), q[2 * u], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              join(widen_lo(w.z, tile.ks), widen_hi(w.z, tile.ks), widen_lo(w.w, tile.ks), widen_hi(w.w, tile.ks)), q[2 * u + 1], acc, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int w = 0; w < kI / 4; ++w)
            v[4 * t + j][w] = reinterpret_cast<const uint32_t*>(tile.v + (4 * g + j) * kD + kI * n)[w];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int w = 0; w < kI / 4; ++w) v[4 * t + j][w] = 0;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = key0 + 4 * g + r;
        const bool see = tile.seen && key < key_hi && key <= pos && (p.window == 0 || pos - key < p.window);
        z[t][r] = see ? acc[r] * p.scale_log2 : kNegInf;
      }
    }
    float top = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])), fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m_new = fmaxf(m, top);
    const float base = m_new == kNegInf ? 0.0f : m_new;
    const float alpha = exp2f(m - base);
    m = m_new;
    l *= alpha;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = exp2f(z[j >> 2][j & 3] - base);
      l += w[j];
    }
    // a NaN value reaches only the rows that see its key: the matrix product
    // would also carry it into rows whose weight is 0
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int i = 0; i < kI / 4; ++i) bad |= nan_bytes(v[j][i]);
    }
    if (__ballot(bad != 0)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < kI / 4; ++i) {
          const uint32_t nb = nan_bytes(v[j][i]);
          hit |= nb;
          v[j][i] &= ~((nb >> 7) * 0xffu);
        }
        const uint64_t who = __ballot(hit != 0);
        if (((who >> (16 * g)) & 0xffffu) && w[j] > 0.0f) l = __builtin_nanf("");
      }
    }
#pragma unroll
    for (int i = 0; i < kI; ++i) o[i] *= alpha;
    const u32x4 pw = {pack2(w[0], w[1]), pack2(w[2], w[3]), pack2(w[4], w[5]), pack2(w[6], w[7])};
    const bf8 pb = __builtin_bit_cast(bf8, pw);
#pragma unroll
    for (int i4 = 0; i4 < kI / 4; ++i4) {
      uint32_t lo[4], hi[4];      // byte pairs (key 2j, key 2j + 1) of two dims each
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = __builtin_amdgcn_perm(v[2 * j + 1][i4], v[2 * j][i4], 0x05010400u);
        hi[j] = __builtin_amdgcn_perm(v[2 * j + 1][i4], v[2 * j][i4], 0x07030602u);
      }
      o[4 * i4 + 0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          join(widen_lo(lo[0], vs[0]), widen_lo(lo[1], vs[0]), widen_lo(lo[2], vs[1]), widen_lo(lo[3], vs[1])), pb, o[4 * i4 + 0], 0, 0, 0);
      o[4 * i4 + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          join(widen_hi(lo[0], vs[0]), widen_hi(lo[1], vs[0]), widen_hi(lo[2], vs[1]), widen_hi(lo[3], vs[1])), pb, o[4 * i4 + 1], 0, 0, 0);
      o[4 * i4 + 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          join(widen_lo(hi[0], vs[0]), widen_lo(hi[1], vs[0]), widen_lo(hi[2], vs[1]), widen_lo(hi[3], vs[1])), pb, o[4 * i4 + 2], 0, 0, 0);
      o[4 * i4 + 3] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          join(widen_hi(hi[0], vs[0]), widen_hi(hi[1], vs[0]), widen_hi(hi[2], vs[1]), widen_hi(hi[3], vs[1])), pb, o[4 * i4 + 3], 0, 0, 0);
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
    sh_m[wave][n] = m;
    sh_l[wave][n] = l;
  }
  __syncthreads();
  const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;   // row and run of kI dims
  if (r0 + jr >= rows) return;
  const int jrow = static_cast<int>(r0) + jr;
  const int jt = p.by_group.div(jrow);
  float top = kNegInf;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sh_m[w][jr]);
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
  f32x4 acc[kI / 4] = {};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = exp2f(sh_m[w][jr] - base);
    sum += f * sh_l[w][jr];
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) acc[i] += f * *reinterpret_cast<const f32x4*>(&sh_o[w][jr][kI * jc + 4 * i]);
  }
  const int64_t at = int64_t(s.row0 + jt) * p.q_heads + h * group + (jrow - jt * group);
  if (p.splits > 1) {
    const int64_t prow = int64_t(blockIdx.x) * c.tokens * p.q_heads + at;
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) *reinterpret_cast<f32x4*>(p.part_o + prow * kD + kI * jc + 4 * i) = acc[i];
    if (jc == 0) {
      p.part_ml[2 * prow] = top;
      p.part_ml[2 * prow + 1] = sum;
    }
    return;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // a NaN sum stays a NaN
#pragma unroll
  for (int i = 0; i < kI / 4; ++i)
    *reinterpret_cast<u32x2*>(p.out + at * kD + kI * jc + 4 * i) =
        u32x2{pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv)};
  if (p.lse && jc == 0) p.lse[at] = (base + log2f(sum)) * kLn2;
}

// Joins the splits: 16 lanes a row, workgroup (16 rows, b).
template <int kD>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams p) {
  constexpr int kI = kD / 16;
  const KvView& c = p.kv;
  const Seq s = load_seq(c, blockIdx.y);
  const int64_t r = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (r >= int64_t(s.n) * p.q_heads) return;
  const int jc = threadIdx.x & 15;
  const int64_t at = int64_t(s.row0) * p.q_heads + r;
  const int64_t pitch = int64_t(c.tokens) * p.q_heads;
  float top = kNegInf;
  for (int k = 0; k < p.splits; ++k) top = fmaxf(top, p.part_ml[2 * (k * pitch + at)]);
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
  f32x4 acc[kI / 4] = {};
  for (int k = 0; k < p.splits; ++k) {
    const int64_t prow = k * pitch + at;
    const float f = exp2f(p.part_ml[2 * prow] - base);
    sum += f * p.part_ml[2 * prow + 1];
#pragma unroll
    for (int i = 0; i < kI / 4; ++i) acc[i] += f * *reinterpret_cast<const f32x4*>(p.part_o + prow * kD + kI * jc + 4 * i);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < kI / 4; ++i)
    *reinterpret_cast<u32x2*>(p.out + at * kD + kI * jc + 4 * i) =
        u32x2{pack2(acc[i].x * inv, acc[i].y * inv), pack2(acc[i].z * inv, acc[i].w * inv)};
  if (p.lse && jc == 0) p.lse[at] = (base + log2f(sum)) * kLn2;
}

// How the keys of a call are split, from its sizes alone.
struct Plan {
  int64_t splits, split_len, row_tiles, workspace;
};
Plan make_plan(const KvView& v, int64_t head_dim, int64_t q_heads, int64_t window) {
  Plan plan{};
  const int64_t group = q_heads / v.heads;
  plan.row_tiles = (int64_t(v.max_new) * group + 15) / 16;
  int64_t span = v.max_len;
  if (window > 0) span = std::min(span, window + 16 + 32);
  span = std::max<int64_t>(span, 1);
  if (plan.row_tiles == 0) return plan;
  const int64_t units = plan.row_tiles * v.batch * v.heads;
  // enough workgroups for four on each of the 256 compute units, of at least 256 keys
  int64_t want = (1024 + units - 1) / units;
  want = std::max<int64_t>(1, std::min(want, span / 256));
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
  if (plan.row_tiles > 65535 || batch->batch * cache->kv_heads > 65535)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: more than 65535 row tiles or (sequence, kv head) pairs", fn);
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
  p.scale_log2 = static_cast<float>(a->softmax_scale * 1.4426950408889634);
  p.q_heads = static_cast<int32_t>(a->q_heads);
  p.window = static_cast<int32_t>(a->window);
  p.splits = static_cast<int32_t>(plan.splits);
  p.split_len = static_cast<int32_t>(plan.split_len);
  p.by_group = FastDiv(static_cast<uint32_t>(a->q_heads / cache->kv_heads));
  const dim3 grid(static_cast<uint32_t>(plan.splits), static_cast<uint32_t>(plan.row_tiles),
                  static_cast<uint32_t>(batch->batch * cache->kv_heads));
  begin_launch();
  if (d == 64) hipLaunchKernelGGL(attend_rows_kernel<64>, grid, dim3(kWaves * 64), 0, stream, p);
  else hipLaunchKernelGGL(attend_rows_kernel<128>, grid, dim3(kWaves * 64), 0, stream, p);
  if (plan.splits > 1) {
    const dim3 jgrid(static_cast<uint32_t>((int64_t(p.kv.max_new) * a->q_heads + 15) / 16), static_cast<uint32_t>(batch->batch));
    if (d == 64) hipLaunchKernelGGL(attend_join_kernel<64>, jgrid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(attend_join_kernel<128>, jgrid, dim3(256), 0, stream, p);
  }
  return check_launch(fn);
}

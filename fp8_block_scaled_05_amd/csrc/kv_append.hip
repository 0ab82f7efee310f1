// Appending keys and values to the paged 8-bit cache, with the norm of each
// head and the position rotation on the way (q too), for gfx950.
//
// One launch.  A workgroup of the first part owns one page's new tokens of
// one kv head, for k or for v: all of a page's rows meet in its registers, so
// the page's amax, its power-of-two scale and the codes need one read of the
// input.  Where the page held older tokens and its scale grows, the same
// workgroup rewrites them.  The other workgroups norm and rotate rows of q.
// Bound by memory: 2 bytes in and out per element of q, 2 in and 1 out per
// element of k and v (six prompts, 14647 tokens with 64 + 2 * 8 heads of 128:
// 115 us, 5.0 TB/s); with a token a sequence by the latency of table, input and
// cache one after the other (33 sequences: 4.9 us).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kv_common.hpp"
#include "kv_slots.hpp"

namespace fp8bs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kMinExp = -32;       // the smallest exponent of a page's scale
constexpr int kQPasses = 4;        // rows of q that a lane has in flight
static_assert(256 / (64 / 8) * kQPasses == 1 << 7 && 256 / (128 / 8) * kQPasses == 1 << 6, "rows of q of a workgroup");

struct AppendParams {
  KvView kv;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  const float* rope;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  int64_t ld_q, hs_q, ld_k, hs_k, ld_v, hs_v;
  float eps;
  int32_t q_heads;
  int32_t rope_rows;
  int32_t rot;
  int32_t kv_blocks;     // workgroups of pages: slots * kv_heads * 2
  Slots pages, queries;
  FastDiv by_q_heads, by_kv2;
};

struct LaneBallot {
  template <class F>
  __device__ __forceinline__ uint64_t ballot(F f) const { return __ballot(f(static_cast<int>(threadIdx.x & 63))); }
};
// Sequence and part of slot i; false: there is none.
__device__ __forceinline__ bool locate(const KvView& c, const Slots& s, int32_t i, int32_t& b, int32_t& part) {
  if (s.search) return find_slot(LaneBallot{}, c, s, i, b, part);
  b = s.by_parts.div(i);
  part = i - b * s.by_parts.d;
  return true;
}

// Eight bf16 of one row.
struct Eight {
  float x[8];
};
__device__ __forceinline__ Eight widen8(u32x4 u) {
  return Eight{{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y), bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)}};
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// Sum over the kL lanes that hold one row.
template <int kL>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = kL / 2; d; d >>= 1) v += __shfl_xor(v, d, kL);
  return v;
}

// What a lane keeps for its eight columns over all its rows.
template <int kL, bool kHalf>
struct Turn {
  int col;            // first column
  bool turned;        // its columns are in the rotated part
  bool second;        // half layout: it holds the second of the pairs
  int partner;        // half layout: lane (within the row) with the other of the pairs
  __device__ __forceinline__ Turn(int lane, int rot) {
    col = lane * 8;
    turned = col < rot;
    second = kHalf && col >= rot / 2;
    partner = turned ? (second ? lane - rot / 16 : lane + rot / 16) : lane;
  }
  // y = rotated x; angles: the position's row of the table.
  __device__ __forceinline__ void apply(Eight& e, const float* angles, int rot) const {
    if constexpr (kHalf) {
      float other[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = __shfl(e.x[i], partner, kL);
      if (turned) {
        const float* c = angles + (second ? col - rot / 2 : col);
        const float* s = c + rot / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float b = other[i] * s[i];
          e.x[i] = second ? __builtin_fmaf(e.x[i], c[i], b) : __builtin_fmaf(e.x[i], c[i], -b);
        }
      }
    } else {
      if (turned) {
        const float* c = angles + col / 2;
        const float* s = c + rot / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = e.x[2 * i], b = e.x[2 * i + 1];
          e.x[2 * i] = __builtin_fmaf(a, c[i], -(b * s[i]));
          e.x[2 * i + 1] = __builtin_fmaf(b, c[i], a * s[i]);
        }
      }
    }
  }
};

// The smallest e >= kMinExp with amax <= 448 * 2^e: with amax = m 2^x,
// 0.5 <= m < 1, that is x - 9, or x - 8 where m > 448 / 512.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = int(u >> 23) - 126;
  const int e = x - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(uint32_t(clamp_i(e, -126, 127) + 127) << 23); }

template <int kD, int kPasses, bool kHalf>
__device__ __forceinline__ void append_page(const AppendParams& p, int block) {
  constexpr int kL = kD / 8;           // lanes of a row
  constexpr int kRows = 256 / kL;      // rows of a pass
  __shared__ float red[4];
  const KvView& c = p.kv;
  const uint32_t rest = p.by_kv2.div(block);
  const int hk = block - rest * p.by_kv2.d;
  int b, chunk;
  if (!locate(c, p.pages, rest, b, chunk)) return;
  const int h = hk >> 1;
  const bool is_k = (hk & 1) == 0;
  const Seq s = load_seq(c, b);
  const int first = s.start > 0 ? s.start : 0;
  const int page_i = (first >> c.page_shift) + chunk;
  const int base = page_i << c.page_shift;
  const int p0 = max(first, base);
  int stop = min(s.end, s.start + s.n);
  if (p.rot) stop = min(stop, p.rope_rows);
  const int p1 = min(stop, base + (1 << c.page_shift));
  if (p0 >= p1) return;
  const int page = c.table[b * c.ld_table + page_i];
  if (page < 0 || page >= c.pages) return;

  const int lane = threadIdx.x % kL, row = threadIdx.x / kL;
  const int64_t slot = int64_t(page) * c.heads + h;
  float* scale_at = (is_k ? c.k_scale : c.v_scale) + slot;
  uint8_t* codes = (is_k ? c.k : c.v) + ((slot << c.page_shift) * kD) + lane * 8;
  const int off = p0 - base, count = p1 - p0;
  const int64_t ld = is_k ? p.ld_k : p.ld_v;
  const uint16_t* src = (is_k ? p.k : p.v) + int64_t(s.row0 + (p0 - s.start)) * ld + h * (is_k ? p.hs_k : p.hs_v) + lane * 8;
  const float old_scale = off ? *scale_at : 0.0f;

  Eight y[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row;
    y[i] = r < count ? widen8(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + r * ld))) : Eight{};
  }
  float amax = 0.0f;
  if (is_k && (p.k_weight || p.rot)) {
    const Turn<kL, kHalf> turn(lane, p.rot);
    Eight w{};
    if (p.k_weight) w = widen8(*reinterpret_cast<const u32x4*>(p.k_weight + lane * 8));
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (i * kRows >= count) break;
      const int r = min(i * kRows + row, count - 1);
      if (p.k_weight) {
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(y[i].x[j], y[i].x[j], sq);
        const float inv = rsqrtf(row_sum<kL>(sq) * (1.0f / kD) + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i].x[j] = y[i].x[j] * inv * w.x[j];
      }
      if (p.rot) turn.apply(y[i], p.rope + int64_t(p0 + r) * p.rot, p.rot);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[i].x[j]));
  }
  amax = wave_max(amax);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));

  int e = scale_exponent(amax);
  if (off) {
    const int e_old = int(__float_as_uint(old_scale) >> 23 & 0xff) - 127;
    if (e_old >= e) {
      e = e_old;
    } else {
      const float shrink = exp2i(e_old - e);
      for (int r = row; r < off; r += kRows) {
        u32x2* at = reinterpret_cast<u32x2*>(codes + r * kD);
        u32x2 was = *at;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int word = static_cast<int>(was[j]);
          const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
          const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
          was[j] = pack4_e4m3(lo[0] * shrink, lo[1] * shrink, hi[0] * shrink, hi[1] * shrink);
        }
        *at = was;
      }
    }
  }
  if (threadIdx.x == 0) *scale_at = exp2i(e);
  const float inv = exp2i(-e);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row;
    if (r < count) {
      const Eight& z = y[i];
      *reinterpret_cast<u32x2*>(codes + (off + r) * kD) =
          u32x2{pack4_e4m3(z.x[0] * inv, z.x[1] * inv, z.x[2] * inv, z.x[3] * inv),
                pack4_e4m3(z.x[4] * inv, z.x[5] * inv, z.x[6] * inv, z.x[7] * inv)};
    }
  }
}

// Rows of q: row r of a sequence is head r % q_heads of its new token
// r / q_heads, so that consecutive rows share their angles.
template <int kD, bool kHalf>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int block) {
  constexpr int kL = kD / 8;
  constexpr int kRows = 256 / kL;
  int b, part;
  if (!locate(p.kv, p.queries, block, b, part)) return;
  const Seq s = load_seq(p.kv, b);
  const int64_t rows = int64_t(s.n) * p.q_heads;
  const int64_t r0 = int64_t(part) * (kRows * kQPasses);
  if (r0 >= rows) return;
  const int lane = threadIdx.x % kL;
  const Turn<kL, kHalf> turn(lane, p.rot);
  Eight w{};
  if (p.q_weight) w = widen8(*reinterpret_cast<const u32x4*>(p.q_weight + lane * 8));
  int token[kQPasses], head[kQPasses];
  u32x4 raw[kQPasses];
#pragma unroll
  for (int i = 0; i < kQPasses; ++i) {
    const uint32_t r = static_cast<uint32_t>(min(r0 + i * kRows + threadIdx.x / kL, rows - 1));
    token[i] = p.by_q_heads.div(r);
    head[i] = r - token[i] * p.by_q_heads.d;
    raw[i] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(p.q + int64_t(s.row0 + token[i]) * p.ld_q + head[i] * p.hs_q + lane * 8));
  }
#pragma unroll
  for (int i = 0; i < kQPasses; ++i) {
    Eight y = widen8(raw[i]);
    if (p.q_weight) {
      float sq = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(y.x[j], y.x[j], sq);
      const float inv = rsqrtf(row_sum<kL>(sq) * (1.0f / kD) + p.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) y.x[j] = y.x[j] * inv * w.x[j];
    }
    if (p.rot) {
      const int pos = s.start + token[i];
      const bool placed = pos >= 0 && pos < p.rope_rows;
      turn.apply(y, p.rope + int64_t(placed ? pos : 0) * p.rot, p.rot);
      if (!placed) y = Eight{};
    }
    if (r0 + i * kRows + threadIdx.x / kL < rows) {
      const int64_t at = (int64_t(s.row0 + token[i]) * p.q_heads + head[i]) * kD + lane * 8;
      __builtin_nontemporal_store(u32x4{pack2(y.x[0], y.x[1]), pack2(y.x[2], y.x[3]), pack2(y.x[4], y.x[5]), pack2(y.x[6], y.x[7])},
                                  reinterpret_cast<u32x4*>(p.q_out + at));
    }
  }
}

template <int kD, int kPasses, bool kHalf>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendParams p) {
  const int block = blockIdx.x;
  if (block < p.kv_blocks) append_page<kD, kPasses, kHalf>(p, block);
  else turn_queries<kD, kHalf>(p, block - p.kv_blocks);
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" fp8bs_status fp8_kv_append(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch, const fp8bs_kv_append_args* a,
                                      hipStream_t stream) {
  const char* fn = "fp8_kv_append";
  AppendParams p{};
  if (!a) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  if (fp8bs_status st = check_kv(fn, cache, batch, true, &p.kv)) return st;
  const int64_t d = cache->head_dim, t = batch->tokens;
  if (a->q_heads < 0 || a->q_heads > 65535) return fail(FP8BS_ERR_INVALID_ARG, "%s: q_heads %lld out of range", fn, (long long)a->q_heads);
  if (a->rot < 0 || a->rot > d || a->rot % 16)
    return fail(FP8BS_ERR_SHAPE, "%s: rot %lld is not a multiple of 16 in 0 .. head_dim", fn, (long long)a->rot);
  if (a->rope_layout != FP8BS_ROPE_HALF && a->rope_layout != FP8BS_ROPE_INTERLEAVED)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown rope_layout %lld", fn, (long long)a->rope_layout);
  if (!(a->eps >= 0.0 && a->eps <= 1e6)) return fail(FP8BS_ERR_INVALID_ARG, "%s: eps %g out of range", fn, a->eps);
  if (a->rot && (a->rope_rows < 1 || a->rope_rows >= (int64_t(1) << 31)))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: rope_rows %lld out of range", fn, (long long)a->rope_rows);
  if (t == 0) return FP8BS_OK;
  if (a->rot && !a->rope) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (rope)", fn);
  if (fp8bs_status st = check_rows(fn, "k", a->k, t, cache->kv_heads, d, a->ld_k, a->hs_k)) return st;
  if (fp8bs_status st = check_rows(fn, "v", a->v, t, cache->kv_heads, d, a->ld_v, a->hs_v)) return st;
  if (a->q_heads) {
    if (fp8bs_status st = check_rows(fn, "q", a->q, t, a->q_heads, d, a->ld_q, a->hs_q)) return st;
    if (fp8bs_status st = check_rows(fn, "q_out", a->q_out, t, a->q_heads, d, a->q_heads * d, d)) return st;
  }
  if (!aligned16(a->rope) || !aligned16(a->q_weight) || !aligned16(a->k_weight))
    return fail(FP8BS_ERR_ALIGNMENT, "%s: rope and weights must be 16-byte aligned", fn);

  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.rope = a->rope;
  p.q_weight = static_cast<const uint16_t*>(a->q_weight);
  p.k_weight = static_cast<const uint16_t*>(a->k_weight);
  p.ld_q = a->ld_q; p.hs_q = a->hs_q; p.ld_k = a->ld_k; p.hs_k = a->hs_k; p.ld_v = a->ld_v; p.hs_v = a->hs_v;
  p.eps = static_cast<float>(a->eps);
  p.q_heads = static_cast<int32_t>(a->q_heads);
  p.rope_rows = static_cast<int32_t>(a->rot ? a->rope_rows : 0);
  p.rot = static_cast<int32_t>(a->rot);
  const int64_t size = cache->page_size;
  const int64_t rows = int64_t(p.kv.max_new) * a->q_heads;
  if (rows >= (int64_t(1) << 31)) return fail(FP8BS_ERR_INVALID_ARG, "%s: 2^31 or more rows of a sequence", fn);
  const int q_shift = d == 64 ? 7 : 6;           // rows of q of a workgroup: 256 / (d / 8) * kQPasses
  int64_t page_slots = 0, query_slots = 0;
  p.pages = Slots::make(p.kv, 1, p.kv.page_shift, 2, (p.kv.max_new + size - 2) / size + 1, &page_slots);
  if (a->q_heads) p.queries = Slots::make(p.kv, a->q_heads, q_shift, 1, (rows + (int64_t(1) << q_shift) - 1) >> q_shift, &query_slots);
  const int64_t kv_blocks = page_slots * cache->kv_heads * 2;
  if (kv_blocks + query_slots >= (int64_t(1) << 24)) return fail(FP8BS_ERR_INVALID_ARG, "%s: 2^24 or more workgroups", fn);
  p.kv_blocks = static_cast<int32_t>(kv_blocks);
  p.by_q_heads = FastDiv(static_cast<uint32_t>(std::max<int64_t>(a->q_heads, 1)));
  p.by_kv2 = FastDiv(static_cast<uint32_t>(cache->kv_heads * 2));
  const dim3 grid(static_cast<uint32_t>(kv_blocks + query_slots));
  const bool half = a->rope_layout == FP8BS_ROPE_HALF;
  // a pass of a page's workgroup is 256 * 8 elements
  const int64_t passes = (std::min<int64_t>(size, p.kv.max_new) * d + 2047) / 2048;
  begin_launch();
#define FP8BS_L(D, N) \
  do { \
    if (half) hipLaunchKernelGGL((kv_append_kernel<D, N, true>), grid, dim3(256), 0, stream, p); \
    else hipLaunchKernelGGL((kv_append_kernel<D, N, false>), grid, dim3(256), 0, stream, p); \
  } while (0)
#define FP8BS_D(D) \
  do { \
    if (passes <= 1) FP8BS_L(D, 1); \
    else if (passes <= 2) FP8BS_L(D, 2); \
    else if (passes <= 4) FP8BS_L(D, 4); \
    else FP8BS_L(D, 8); \
  } while (0)
  if (d == 64) FP8BS_D(64); else FP8BS_D(128);
#undef FP8BS_D
#undef FP8BS_L
  return check_launch(fn);
}

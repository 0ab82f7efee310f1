// What the kernels of the paged cache share: the batch as a kernel sees it,
// and the host checks of its sizes.
#pragma once
#include <hip/hip_runtime.h>
#include <algorithm>
#include <cstdint>

#include "device.hpp"
#include "fp8bs_decoder.h"
#include "status.hpp"

namespace fp8bs {

struct KvView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int64_t ld_table;
  int32_t width;       // pages in a row of the block table
  int32_t pages;
  int32_t heads;       // kv heads
  int32_t page_shift;  // page size = 1 << page_shift
  int32_t batch;
  int32_t tokens;
  int32_t max_new;
  int32_t max_len;
};

// Rows and positions of one sequence, from tables that may hold anything:
// rows [row0, row0 + n) lie in [0, tokens), n <= max_new.  The position of
// row row0 + i is start + i.  end is one past the last position that may be
// read or written: within the table's row and max_len.
struct Seq {
  int32_t row0, n, start, end;
};
__host__ __device__ __forceinline__ int32_t clamp_i(int32_t v, int32_t lo, int32_t hi) { return v < lo ? lo : (v > hi ? hi : v); }
__host__ __device__ __forceinline__ Seq make_seq(int32_t cu0, int32_t cu1, int32_t len, int32_t tokens, int32_t max_new,
                                                 int32_t max_len, int32_t width, int32_t page_shift) {
  Seq s;
  s.row0 = clamp_i(cu0, 0, tokens);
  const int32_t n = clamp_i(cu1, s.row0, tokens) - s.row0;
  len = clamp_i(len, 0, 1 << 30);
  s.start = len - n;
  s.n = n < max_new ? n : max_new;
  const int64_t room = int64_t(width) << page_shift;
  int64_t end = len < max_len ? len : max_len;
  end = end < room ? end : room;
  s.end = end > 0 ? static_cast<int32_t>(end) : 0;
  return s;
}
__host__ __device__ __forceinline__ Seq load_seq(const KvView& c, int b) {
  return make_seq(c.cu[b], c.cu[b + 1], c.lens[b], c.tokens, c.max_new, c.max_len, c.width, c.page_shift);
}

inline bool mul_fits(int64_t a, int64_t b, int64_t limit) { return a == 0 || b <= limit / a; }

// Sizes and pointers of a cache and a batch.  `pointers` false: sizes only.
inline fp8bs_status check_kv(const char* fn, const fp8bs_kv_cache* c, const fp8bs_kv_batch* b, bool pointers, KvView* view) {
  if (!c || !b) return fail(FP8BS_ERR_INVALID_ARG, "%s: null argument struct", fn);
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (c->pages < 0 || c->pages > lim || c->kv_heads < 1 || c->kv_heads > 65535)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: pages %lld, kv_heads %lld out of range", fn, (long long)c->pages, (long long)c->kv_heads);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(FP8BS_ERR_SHAPE, "%s: page_size %lld is not 16, 32, 64 or 128", fn, (long long)c->page_size);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(FP8BS_ERR_SHAPE, "%s: head_dim %lld is not 64 or 128", fn, (long long)c->head_dim);
  if (!mul_fits(c->pages * c->kv_heads, c->page_size * c->head_dim, kMaxBytes))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: cache larger than any allocation", fn);
  if (b->batch < 1 || b->batch > 65535 || b->tokens < 0 || b->tokens > (1 << 30) || b->table_width < 0 || b->table_width > lim ||
      b->max_new < 0 || b->max_new > lim || b->max_len < 0 || b->max_len > (1 << 30))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: batch %lld, tokens %lld, table_width %lld, max_new %lld or max_len %lld out of range", fn,
                (long long)b->batch, (long long)b->tokens, (long long)b->table_width, (long long)b->max_new, (long long)b->max_len);
  if (b->ld_table < b->table_width || b->ld_table > lim)
    return fail(FP8BS_ERR_INVALID_ARG, "%s: ld_table %lld smaller than the row or out of range", fn, (long long)b->ld_table);
  if (b->tokens > 0 && b->max_new == 0) return fail(FP8BS_ERR_INVALID_ARG, "%s: max_new is 0 with %lld tokens", fn, (long long)b->tokens);
  if (pointers && b->tokens > 0) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !b->cu || !b->seq_lens || !b->block_table)
      return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer in the cache or the batch", fn);
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(FP8BS_ERR_ALIGNMENT, "%s: cache codes must be 16-byte aligned", fn);
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale) || !aligned4(b->cu) || !aligned4(b->seq_lens) || !aligned4(b->block_table))
      return fail(FP8BS_ERR_ALIGNMENT, "%s: scales and index arrays must be 4-byte aligned", fn);
  }
  int shift = 4;
  while ((int64_t(1) << shift) < c->page_size) ++shift;
  *view = KvView{c->k, c->v, c->k_scale, c->v_scale, b->cu, b->seq_lens, b->block_table, b->ld_table,
                 static_cast<int32_t>(b->table_width), static_cast<int32_t>(c->pages), static_cast<int32_t>(c->kv_heads), shift,
                 static_cast<int32_t>(b->batch), static_cast<int32_t>(b->tokens),
                 static_cast<int32_t>(std::min(b->max_new, b->tokens)), static_cast<int32_t>(b->max_len)};
  return FP8BS_OK;
}

// Rows [tokens, heads, head_dim] of bf16 with pitches in elements.
inline fp8bs_status check_rows(const char* fn, const char* what, const void* p, int64_t tokens, int64_t heads, int64_t dim,
                               int64_t ld, int64_t hs) {
  if (!p) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (%s)", fn, what);
  if (ld < 0 || hs < 0 || ld > kMaxExtent || hs > kMaxExtent || !mul_fits(std::max<int64_t>(ld, 1), tokens, kMaxBytes / 2) ||
      !mul_fits(std::max<int64_t>(hs, 1), heads, kMaxBytes / 2))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: pitches of %s exceed any allocation", fn, what);
  if ((heads > 1 && hs < dim) || (tokens > 1 && ld < dim))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch of %s smaller than head_dim", fn, what);
  if (!aligned16(p) || ld % 8 || hs % 8)
    return fail(FP8BS_ERR_ALIGNMENT, "%s: %s and its pitches must be 16-byte aligned", fn, what);
  return FP8BS_OK;
}

}  // namespace fp8bs

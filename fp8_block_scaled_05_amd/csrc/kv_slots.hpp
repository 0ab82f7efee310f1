// How append's workgroups find their sequence.
//
// A sequence's work (its pages, its rows of q) falls into parts.  Where the
// sequences are alike, workgroup i takes part i % parts of sequence i / parts,
// with as many parts as the longest may have.  One prompt among many single
// tokens would leave most of those workgroups without work (and need 2^25 of
// them for 1024 sequences with one prompt of 16384 tokens), so there the parts
// are numbered over all sequences: sequence b's begin at
//   base(b) = floor(cu[b] * per_token / 2^shift) + spare * b,
// which leaves at least floor(n * per_token / 2^shift) + spare of them for its
// n tokens, and a wave finds b by looking at 64 sequences at once.  `Wave`
// gives the ballot of a function over the 64 lanes, so that the same code runs
// on the host.
#pragma once
#include "kv_common.hpp"

namespace fp8bs {

struct Slots {
  int32_t search;        // parts are numbered over all sequences
  int32_t per_token;
  int32_t shift, spare;
  FastDiv by_parts;      // else: parts of every sequence

  // `parts` of the longest sequence.  The search costs a workgroup a load and
  // is taken where it saves two of three: one prompt of 8192 tokens among
  // single ones, 64 + 2 * 8 heads of 128, in 3 sequences 68.8 us (without
  // 68.3), in 4 67.5 (70.1), in 8 67.0 (81.7), in 64 74 (253), in 256 93 (844);
  // six prompts, 14647 tokens of which the longest has 4096, 118 us (115).
  static Slots make(const KvView& c, int64_t per_token, int32_t shift, int32_t spare, int64_t parts, int64_t* total) {
    const int64_t alike = c.batch * parts, packed = ((c.tokens * per_token) >> shift) + int64_t(spare) * c.batch;
    const bool search = 3 * packed < alike;
    *total = search ? packed : alike;
    return {search, static_cast<int32_t>(per_token), shift, spare, FastDiv(static_cast<uint32_t>(std::max<int64_t>(parts, 1)))};
  }
  __host__ __device__ __forceinline__ int32_t base(const KvView& c, int32_t b) const {
    return static_cast<int32_t>((int64_t(clamp_i(c.cu[b], 0, c.tokens)) * per_token) >> shift) + spare * b;
  }
};

// Sequence and part of workgroup i where parts are numbered over all
// sequences.  cu may hold anything: b lies in the batch, and part is not
// negative, in any case.
template <class Wave>
__host__ __device__ __forceinline__ bool find_slot(const Wave& wave, const KvView& c, const Slots& s, int32_t i, int32_t& b, int32_t& part) {
  int32_t lo = 0, hi = c.batch;          // the last b with base(b) <= i
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 63) >> 6;
    const uint64_t below = wave.ballot([&](int lane) {
      const int32_t at = lo + lane * step;
      return at < hi && s.base(c, at < hi ? at : lo) <= i;
    });
    const int many = __builtin_popcountll(below);
    lo += (many ? many - 1 : 0) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  b = lo;
  part = i - s.base(c, lo);
  return part >= 0;
}

}  // namespace fp8bs

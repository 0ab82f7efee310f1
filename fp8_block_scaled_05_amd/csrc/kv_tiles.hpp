// The order of attention's 128-row tiles over all sequences of a batch.
//
// The i-th tile, those at later positions first: they see more keys, and
// started last they would run on alone.  A tile's place is its first row's
// position in units of 128 rows, so the place that holds the i-th tile is
// found by bisection over counts (sequence by sequence two prompts, of 8192
// tokens and of 2179 over 6522, took 867 us and not 795).  Every wave does it by itself, with a
// sequence a lane; `Wave` gives the sum and the ballot of a function over the
// 64 lanes, so that the same code runs on the host.
//
// cu may hold anything (then sequences may claim the same rows, and tiles may
// number far more than rows).  What is returned is a sequence of the batch and
// a tile of it.
#pragma once
#include "kv_common.hpp"

namespace fp8bs {

struct TilePlace {
  int32_t place, n;    // of a sequence: its first tile's place, its tiles
};
__host__ __device__ __forceinline__ TilePlace tile_place(const KvView& c, int b, int group) {
  if (b >= c.batch) return {0, 0};
  const Seq s = load_seq(c, b);
  const int64_t place = (int64_t(s.start > 0 ? s.start : 0) * group) >> 7, most = int64_t(1) << 29;
  return {static_cast<int32_t>(place < most ? place : most), static_cast<int32_t>((int64_t(s.n) * group + 127) >> 7)};
}
__host__ __device__ __forceinline__ int32_t tiles_from(TilePlace t, int32_t from) { return clamp_i(t.place + t.n - from, 0, t.n); }

// More tiles than a call may have (attention refuses 2^23).
constexpr int32_t kManyTiles = 1 << 24;
__host__ __device__ __forceinline__ int32_t fewer(int32_t a, int32_t b) { return a < b ? a : b; }

// i < kManyTiles.
template <class Wave>
__host__ __device__ __forceinline__ bool find_tile(const Wave& wave, const KvView& c, int i, int group, int& seq, int& tile) {
  // Tiles at `from` and later, where they are fewer than kManyTiles; else at
  // least that many: a lane's sum stops there, and 64 lanes stay below 2^31.
  auto count = [&](int from) {
    return wave.sum([&](int lane, TilePlace first) {
      int sum = tiles_from(first, from);          // at most 2^24
      for (int b = 64 + lane; b - lane < c.batch; b += 64) sum = fewer(sum + tiles_from(tile_place(c, b, group), from), kManyTiles);
      return sum;
    });
  };
  if (count(0) <= i) return false;
  int lo = 0, hi = 1, above = 0;         // count(lo) > i >= count(hi) = above
  for (;;) {
    const int n = count(hi);
    if (n <= i) {
      above = n;
      break;
    }
    lo = hi;
    hi *= 2;
  }
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2, n = count(mid);
    if (n > i) lo = mid;
    else { hi = mid; above = n; }
  }
  int left = i - above;                  // which of the tiles at `lo`
  for (int b0 = 0; b0 < c.batch; b0 += 64) {
    uint64_t here = wave.ballot([&](int lane, TilePlace first) {
      const TilePlace t = b0 ? tile_place(c, b0 + lane, group) : first;
      return t.place <= lo && lo < t.place + t.n;
    });
    const int many = __builtin_popcountll(here);
    if (left >= many) {
      left -= many;
      continue;
    }
    for (; left; --left) here &= here - 1;
    seq = b0 + __builtin_ctzll(here);
    tile = lo - tile_place(c, seq, group).place;
    return true;
  }
  return false;
}

}  // namespace fp8bs

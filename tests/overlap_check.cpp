// Host run of csrc/overlap.hpp against sets of bytes: compiled by tests/test_overlap.py.  Exit status 0 if every answer is
// right.
#include <cstdio>
#include <random>
#include <set>

#include "overlap.hpp"

using namespace fp8bs;

namespace {

std::set<uintptr_t> bytes(const Block& b) {
  std::set<uintptr_t> s;
  for (int64_t r = 0; b.p && r < b.rows; ++r)
    for (int64_t c = 0; c < b.width; ++c) s.insert(reinterpret_cast<uintptr_t>(b.p) + r * b.pitch + c);
  return s;
}

}  // namespace

int main() {
  std::mt19937 rng(1);
  const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  int met = 0, apart_inside = 0;
  for (int n = 0; n < 200000; ++n) {
    Block b[2];
    const int pitch = pick(1, 24);
    for (Block& x : b) {
      x.pitch = pick(0, 2) ? pitch : pick(1, 24);
      x.width = pick(0, 9) ? pick(1, static_cast<int>(x.pitch)) : x.pitch;
      x.rows = pick(0, 6);
      x.p = pick(0, 40) ? reinterpret_cast<const void*>(uintptr_t(1000 + pick(0, 120))) : nullptr;
    }
    const std::set<uintptr_t> s = bytes(b[0]), t = bytes(b[1]);
    bool want = false;
    for (uintptr_t v : s) want |= t.count(v) != 0;
    if (overlap(b[0], b[1]) != want || overlap(b[1], b[0]) != want) {
      std::printf("%p %ld x %ld / %ld, %p %ld x %ld / %ld: %d\n", b[0].p, long(b[0].rows), long(b[0].width), long(b[0].pitch), b[1].p,
                  long(b[1].rows), long(b[1].width), long(b[1].pitch), want);
      return 1;
    }
    met += want;
    apart_inside += !want && !s.empty() && !t.empty() && *s.begin() <= *t.rbegin() && *t.begin() <= *s.rbegin();
  }
  std::printf("%d meet, %d apart within each other's range\n", met, apart_inside);
  return met > 10000 && apart_inside > 5000 ? 0 : 1;
}

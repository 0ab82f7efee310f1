// Host run of the walks that attention and append take over a batch (csrc/kv_tiles.hpp, csrc/kv_slots.hpp): compiled by
// tests/test_kv_walk.py, for the host only.  Argument: the check's name; exit status 0 if it holds.
#include <cstdio>
#include <cstring>
#include <random>
#include <set>
#include <vector>

#include "kv_slots.hpp"
#include "kv_tiles.hpp"

using namespace fp8bs;

namespace {

struct HostWave {
  TilePlace first[64];
  template <class F>
  int sum(F f) const {
    uint32_t v = 0;                      // wraps as the GPU's additions do
    for (int lane = 0; lane < 64; ++lane) v += static_cast<uint32_t>(f(lane, first[lane]));
    return static_cast<int>(v);
  }
  template <class F>
  uint64_t ballot(F f) const {
    uint64_t m = 0;
    for (int lane = 0; lane < 64; ++lane) m |= uint64_t(f(lane, first[lane]) ? 1 : 0) << lane;
    return m;
  }
};

struct Batch {
  std::vector<int32_t> cu, lens, table;
  KvView view;
  Batch(std::vector<int32_t> cu_, std::vector<int32_t> lens_, int32_t tokens, int32_t max_new, int32_t max_len, int32_t heads, int32_t width,
        int32_t shift)
      : cu(std::move(cu_)), lens(std::move(lens_)) {
    view = KvView{nullptr, nullptr, nullptr, nullptr, cu.data(), lens.data(), nullptr, width, width, 1 << 20, heads, shift,
                  static_cast<int32_t>(lens.size()), tokens, std::min(max_new, tokens), max_len};
  }
};

#define CHECK(cond, ...) \
  do { \
    if (!(cond)) { \
      std::printf("%s: ", #cond); \
      std::printf(__VA_ARGS__); \
      std::printf("\n"); \
      return false; \
    } \
  } while (0)

bool find(const Batch& b, int group, int i, int& seq, int& tile) {
  HostWave w;
  for (int lane = 0; lane < 64; ++lane) w.first[lane] = tile_place(b.view, lane, group);
  return find_tile(w, b.view, i, group, seq, tile);
}
// found tiles are tiles of the batch
bool inside(const Batch& b, int group, int i) {
  int seq = -7, tile = -7;
  if (!find(b, group, i, seq, tile)) return true;
  CHECK(seq >= 0 && seq < b.view.batch, "i %d seq %d", i, seq);
  CHECK(tile >= 0 && tile < tile_place(b.view, seq, group).n, "i %d seq %d tile %d", i, seq, tile);
  return true;
}

// Every tile of a batch is found once, those at later places first.
bool tiles() {
  std::mt19937 rng(1);
  auto draw = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  for (int round = 0; round < 60; ++round) {
    const int batch = draw(1, round % 3 ? 5 : 200), group = draw(1, 9), longest = draw(1, round % 2 ? 30 : 900);
    std::vector<int32_t> cu{0}, lens;
    int max_new = 0, max_len = 0;
    for (int s = 0; s < batch; ++s) {
      const int n = draw(0, 3) ? draw(0, longest) : 0;
      cu.push_back(cu.back() + n);
      lens.push_back(n + draw(0, 2000));
      max_new = std::max(max_new, n);
      max_len = std::max(max_len, lens.back());
    }
    const Batch b(cu, lens, cu.back(), max_new, max_len, 2, 1 << 20, 4);
    int total = 0, last = 1 << 30;
    for (int s = 0; s < batch; ++s) total += tile_place(b.view, s, group).n;
    CHECK(total <= int64_t(cu.back()) * group / 128 + batch, "%d tiles", total);
    std::set<std::pair<int, int>> seen;
    for (int i = 0; i < total; ++i) {
      int seq = -1, tile = -1;
      CHECK(find(b, group, i, seq, tile), "round %d tile %d of %d", round, i, total);
      if (!inside(b, group, i)) return false;
      const int place = tile_place(b.view, seq, group).place + tile;
      CHECK(place <= last, "round %d tile %d: place %d after %d", round, i, place, last);
      last = place;
      CHECK(seen.insert({seq, tile}).second, "round %d seq %d tile %d twice", round, seq, tile);
    }
    int seq, tile;
    CHECK(!find(b, group, total, seq, tile), "round %d: tile %d of %d", round, total, total);
  }
  return true;
}

// cu and seq_lens that hold anything: what is found lies in the batch.
bool crooked_tiles() {
  std::mt19937 rng(2);
  auto draw = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  for (int round = 0; round < 400; ++round) {
    const int batch = draw(1, round % 3 ? 5 : 150), group = draw(1, 9), tokens = draw(1, 5000);
    std::vector<int32_t> cu, lens;
    for (int s = 0; s <= batch; ++s) {
      const int kind = draw(0, 9);
      cu.push_back(kind == 0 ? INT32_MIN : kind == 1 ? INT32_MAX : kind == 2 ? -draw(0, tokens) : draw(0, 2 * tokens));
      if (s < batch) lens.push_back(kind == 3 ? INT32_MIN : kind == 4 ? INT32_MAX : kind == 5 ? -draw(1, 99) : draw(0, 9000));
    }
    const Batch b(cu, lens, tokens, draw(1, tokens), draw(1, 9000), 2, draw(1, 500), 4);
    const int most = int64_t(tokens) * group / 128 + batch;
    for (int i = 0; i < most; i += 1 + most / 50)
      if (!inside(b, group, i)) return false;
  }
  return true;
}

// Each second of 65535 sequences claims all rows: tiles number more than 2^31.
bool many_tiles() {
  for (const int tokens : {1 << 17, 131329, 1 << 18}) {
    const int batch = 65535, group = 64;
    std::vector<int32_t> cu(batch + 1, 0), lens(batch);
    for (int s = 0; s <= batch; ++s) cu[s] = s & 1 ? tokens : 0;
    for (int s = 0; s < batch; ++s) lens[s] = tokens + (s * 7919LL) % 100000;
    const Batch b(cu, lens, tokens, tokens, 1 << 30, 1, 1 << 20, 4);
    const int most = int64_t(tokens) * group / 128 + batch;
    for (const int i : {0, 1, 12345, most / 2, most - 1}) {
      int seq, tile;
      CHECK(find(b, group, i, seq, tile), "i %d of more than %d is not found", i, most);
      if (!inside(b, group, i)) return false;
    }
  }
  return true;
}

struct HostBallot {
  template <class F>
  uint64_t ballot(F f) const {
    uint64_t m = 0;
    for (int lane = 0; lane < 64; ++lane) m |= uint64_t(f(lane) ? 1 : 0) << lane;
    return m;
  }
};
// The pages and the runs of rows that a sequence's new tokens need.
int64_t pages_needed(const KvView& c, int b) {
  const Seq s = load_seq(c, b);
  if (!s.n) return 0;
  const int first = std::max(s.start, 0), last = s.start + s.n - 1;
  return last < first ? 0 : (last >> c.page_shift) - (first >> c.page_shift) + 1;
}

// Every page and every run of rows of a batch has one workgroup, and the launch has no more than both bounds.
bool slots() {
  std::mt19937 rng(3);
  auto draw = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  int searched = 0;
  for (int round = 0; round < 300; ++round) {
    const int batch = draw(1, round % 3 ? 6 : 5000), heads = draw(1, 70), shift = draw(4, 7), q_shift = draw(6, 7);
    std::vector<int32_t> cu{draw(0, 1) * draw(0, 9)}, lens;
    int max_new = 0;
    for (int s = 0; s < batch; ++s) {
      const int kind = draw(0, 9), n = kind == 0 ? 0 : kind == 1 ? draw(1, 700) : round % 2 ? 1 : draw(1, 40);
      cu.push_back(cu.back() + n);
      lens.push_back(n + draw(0, 3) * draw(0, 300));
      max_new = std::max(max_new, n);
    }
    if (!max_new) continue;
    const Batch b(cu, lens, cu.back() + draw(0, 1) * draw(0, 50), max_new, 1 << 20, 2, 1 << 20, shift);
    const int64_t size = 1 << shift, rows = int64_t(b.view.max_new) * heads;
    for (const bool pages : {true, false}) {
      int64_t total;
      const Slots s = pages ? Slots::make(b.view, 1, shift, 2, (b.view.max_new + size - 2) / size + 1, &total)
                            : Slots::make(b.view, heads, q_shift, 1, (rows + (1 << q_shift) - 1) >> q_shift, &total);
      if (!s.search) continue;
      ++searched;
      std::set<std::pair<int, int>> seen;
      for (int i = 0; i < total; ++i) {
        int32_t at, part;
        if (!find_slot(HostBallot{}, b.view, s, i, at, part)) continue;
        CHECK(at >= 0 && at < batch && part >= 0, "slot %d: sequence %d part %d", i, at, part);
        CHECK(seen.insert({at, part}).second, "slot %d: sequence %d part %d twice", i, at, part);
      }
      for (int q = 0; q < batch; ++q) {
        const int64_t need = pages ? pages_needed(b.view, q) : (int64_t(load_seq(b.view, q).n) * heads + (1 << q_shift) - 1) >> q_shift;
        for (int part = 0; part < need; ++part) CHECK(seen.count({q, part}), "sequence %d part %d of %d is not found", q, part, int(need));
      }
    }
  }
  CHECK(searched > 100, "%d", searched);
  return true;
}

// cu that holds anything: a workgroup's sequence lies in the batch.
bool crooked_slots() {
  std::mt19937 rng(4);
  auto draw = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  for (int round = 0; round < 500; ++round) {
    const int batch = draw(1, round % 3 ? 70 : 9000), tokens = draw(1, 5000);
    std::vector<int32_t> cu, lens(batch, 100);
    for (int s = 0; s <= batch; ++s) {
      const int kind = draw(0, 5);
      cu.push_back(kind == 0 ? INT32_MIN : kind == 1 ? INT32_MAX : draw(-tokens, 2 * tokens));
    }
    const Batch b(cu, lens, tokens, tokens, 1000, 2, 64, 4);
    int64_t total;
    const Slots s = Slots::make(b.view, 64, 6, 1, int64_t(tokens), &total);
    for (int i = 0; i < total; i += 1 + static_cast<int>(total / 200)) {
      int32_t at, part;
      if (find_slot(HostBallot{}, b.view, s, i, at, part)) CHECK(at >= 0 && at < batch && part >= 0, "slot %d: sequence %d part %d", i, at, part);
    }
  }
  return true;
}

}  // namespace

int main(int argc, char** argv) {
  const struct { const char* name; bool (*run)(); } checks[] = {{"tiles", tiles}, {"crooked_tiles", crooked_tiles}, {"many_tiles", many_tiles},
                                                               {"slots", slots}, {"crooked_slots", crooked_slots}};
  for (const auto& c : checks)
    if (argc > 1 && !std::strcmp(argv[1], c.name)) return c.run() ? 0 : 1;
  std::printf("no such check\n");
  return 2;
}

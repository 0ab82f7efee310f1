// Host run of the walks that attention and append take over a batch (csrc/kv_tiles.hpp): compiled by
// tests/test_kv_walk.py, for the host only.  Argument: the check's name; exit status 0 if it holds.
#include <cstdio>
#include <cstring>
#include <random>
#include <set>
#include <vector>

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

}  // namespace

int main(int argc, char** argv) {
  const struct { const char* name; bool (*run)(); } checks[] = {{"tiles", tiles}, {"crooked_tiles", crooked_tiles}, {"many_tiles", many_tiles}};
  for (const auto& c : checks)
    if (argc > 1 && !std::strcmp(argv[1], c.name)) return c.run() ? 0 : 1;
  std::printf("no such check\n");
  return 2;
}

// Whether operands of a call share memory (host code only).
#pragma once
#include <cstdint>

namespace fp8bs {

// Rows of `width` bytes, one every `pitch` (>= width).
struct Block {
  const void* p = nullptr;
  int64_t rows = 0, width = 0, pitch = 0;
  bool operator==(const Block& o) const { return p == o.p && rows == o.rows && width == o.width && (pitch == o.pitch || rows <= 1); }
  int64_t extent() const { return (rows - 1) * pitch + width; }
};
inline Block line(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

namespace detail {

// Whether a row of `b` meets [lo, hi), relative to b's first byte.
inline bool meets(const Block& b, int64_t lo, int64_t hi) {
  const int64_t i = lo < b.width ? 0 : (lo - b.width) / b.pitch + 1;       // the first row that ends behind lo
  return i < b.rows && i * b.pitch < hi;
}

// Of blocks whose ranges of addresses meet, b's first byte d behind a's.
inline bool rows_meet(Block a, Block b, int64_t d) {
  for (Block* x : {&a, &b})
    if (x->rows == 1 || x->pitch == x->width) *x = line(x->p, x->rows * x->width);
  if (b.rows == 1) return meets(a, d, d + b.width);
  if (a.rows == 1) return meets(b, -d, -d + a.width);
  if (a.pitch == b.pitch) {
    // b's row j begins `in` bytes into the pitch of a's row j + q, and may reach
    // into that of the next one.
    const int64_t q = d >= 0 ? d / a.pitch : -((-d + a.pitch - 1) / a.pitch), in = d - q * a.pitch;
    const auto same_rows = [&](int64_t first) { return first < a.rows && first + b.rows > 0; };
    return (in < a.width && same_rows(q)) || (in + b.width > a.pitch && same_rows(q + 1));
  }
  // Rows of different pitches: each of the fewer ones by itself.
  const bool fewer_a = a.rows <= b.rows;
  const Block &few = fewer_a ? a : b, &many = fewer_a ? b : a;
  const int64_t at = fewer_a ? -d : d;
  for (int64_t i = 0; i < few.rows; ++i)
    if (meets(many, at + i * few.pitch, at + i * few.pitch + few.width)) return true;
  return false;
}

}  // namespace detail

// Whether the two share a byte.  Exact: two halves of one matrix do not, though
// their ranges of addresses do.
inline bool overlap(const Block& a, const Block& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  return d < a.extent() && -d < b.extent() && detail::rows_meet(a, b, d);
}

}  // namespace fp8bs

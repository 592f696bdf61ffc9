// Checks of strides, alignment and overlapping arguments, shared by the
// training and block entry points (api_train.cpp, api_block.cpp). Host only.
#pragma once

#include <stdint.h>

#include <initializer_list>
#include <utility>

namespace moe {

constexpr int64_t kMaxElements = (int64_t)1 << 60;  // rows * stride at most: byte offsets fit 64 bits

// `rows` rows of `width` bytes, `ld` bytes apart, from p.
struct Range {
  const void* p;
  int64_t width;
  int64_t rows = 1, ld = 0;
};

// `rows` rows of `width` elements, `ld` elements apart.
inline Range span(const void* p, int64_t rows, int64_t ld, int64_t width, int64_t bytes) {
  if (rows <= 1 || ld == width) return {p, rows * width * bytes};
  return {p, width * bytes, rows, ld * bytes};
}

// a and b share a byte. Exact for blocks and for rows of equal strides; rows
// of unequal strides count as sharing one where their first-to-last bytes do.
// (Null and empty ranges share none.)
inline bool share(Range a, Range b) {
  uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x == 0 || y == 0 || a.width <= 0 || b.width <= 0) return false;
  if (y < x) {
    std::swap(a, b);
    std::swap(x, y);
  }
  const uint64_t off = y - x;  // b starts at this byte of a's
  if (off >= (uint64_t)((a.rows - 1) * a.ld + a.width)) return false;
  if (a.rows == 1 || (b.rows > 1 && b.ld != a.ld)) return true;
  // b's first row starts in a row of a or in the gap behind one; a further row
  // of a follows that gap, so b has to end before it. b's other rows, at the
  // same stride, repeat this.
  const uint64_t at = off % (uint64_t)a.ld;
  return at < (uint64_t)a.width || at + (uint64_t)b.width > (uint64_t)a.ld;
}

// One of `outs` shares a byte with another of them or with one of `ins`.
inline bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* a = outs.begin(); a != outs.end(); ++a) {
    for (const Range* b = a + 1; b != outs.end(); ++b)
      if (share(*a, *b)) return true;
    for (const Range& b : ins)
      if (share(*a, b)) return true;
  }
  return false;
}

// A row stride that does not cover `width`, is no multiple of `multiple`, or
// takes `rows` rows past kMaxElements.
inline bool bad_ld(int64_t ld, int64_t width, int64_t multiple, int64_t rows) {
  return ld < width || ld % multiple != 0 || ld > kMaxElements / (rows > 1 ? rows : 1);
}

inline bool misaligned(const void* p, uintptr_t to) { return (uintptr_t)p % to != 0; }

}  // namespace moe

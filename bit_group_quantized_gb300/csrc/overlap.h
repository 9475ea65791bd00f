// overlap.h — whether two strided arrays have bytes in common. Plain C++, so
// that the host can check it as the entry points run it.
#pragma once

#include <stdint.h>

#include <initializer_list>
#include <numeric>

namespace bgq {

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* at;
  int64_t rows, width, stride;  // width at most stride
};

// Rows of one array may lie between the other's. Where the bytes from the first row's first to the last row's last meet, rows i and j
// are a distance apart that leaves d after division by what both strides are multiples of, and any such distance counts as one
// that occurs: exact where both strides are the same, and refusing a little more where they are not.
inline bool overlap(const Rows& a, const Rows& b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  const uint64_t pa = (uint64_t)(uintptr_t)a.at, pb = (uint64_t)(uintptr_t)b.at;
  const uint64_t sa = (uint64_t)(a.rows - 1) * a.stride + a.width, sb = (uint64_t)(b.rows - 1) * b.stride + b.width;
  if (pa < pb ? pb - pa >= sa : pa - pb >= sb) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  // an array of one row has any stride: the other's
  const uint64_t g = a.rows == 1 ? b.stride : b.rows == 1 ? a.stride : std::gcd((uint64_t)a.stride, (uint64_t)b.stride);
  const uint64_t d = pa < pb ? (pb - pa) % g : (g - (pa - pb) % g) % g;  // b's rows begin d behind a's
  return d < (uint64_t)a.width || d + b.width > g;
}

// One of `written` meets another of them, or one of `read`.
inline bool overlap(std::initializer_list<Rows> written, std::initializer_list<Rows> read) {
  for (const Rows* w = written.begin(); w != written.end(); ++w) {
    for (const Rows* v = written.begin(); v != w; ++v)
      if (overlap(*w, *v)) return true;
    for (const Rows& r : read)
      if (overlap(*w, r)) return true;
  }
  return false;
}

}  // namespace bgq

// What the entry points check of pointers: alignment, presence, overlaps.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdn {

inline size_t align_up(size_t n) { return (n + 255) / 256 * 256; }
inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <typename... P> bool all_aligned(P... p) { return (aligned(p) && ...); }
template <typename... P> bool all_given(P... p) { return (... && (p != nullptr)); }

// A tensor's bytes; whether any of the outputs shares some with any input or other output.
struct Range {
  const void* p;
  size_t n;
};
inline bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
template <int NO, int NI> bool overlaps(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

}  // namespace gdn

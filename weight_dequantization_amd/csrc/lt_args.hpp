// lt_args.hpp -- host-side argument checks that liblt's entry points share.
#pragma once
#include <stdint.h>

namespace lt {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// rows*cols elements in groups of `group`; see lt.h for the rule.
inline bool shape_ok(uint64_t rows, uint64_t cols, uint64_t group) {
  if (rows == 0 || cols == 0 || group == 0) return false;
  if (rows > (~0ull) / cols) return false;
  uint64_t n = rows * cols;
  if (n > (1ull << 48)) return false;
  if (cols % group != 0 && group % cols != 0) return false;
  if (n % group != 0) return false;
  return true;
}

inline uint32_t shift_of(uint64_t g) {
  return (g & (g - 1)) == 0 ? (uint32_t)__builtin_ctzll(g) : 64u;
}

}  // namespace lt

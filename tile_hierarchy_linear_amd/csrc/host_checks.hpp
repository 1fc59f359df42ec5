// host_checks.hpp -- argument checks shared by the C entry points (host code
// only): element sizes, byte ranges and their overlap.
#pragma once

#include <stdint.h>

#include "../../include/thl.h"

namespace thl {

// Bytes of `count` elements of a format (4-bit: two per byte, rounded up).
inline int64_t bytes_of(thl_dtype t, int64_t count) {
  switch (t) {
    case THL_F32:
    case THL_I32:
      return 4 * count;
    case THL_F16:
    case THL_BF16:
      return 2 * count;
    case THL_I8:
    case THL_E4M3:
    case THL_E5M2:
    case THL_E8M0:
      return count;
    case THL_E2M1X2:
    case THL_I4X2:
    case THL_U4X2:
      return (count + 1) / 2;
    case THL_E2M3:
    case THL_E3M2:
      return (6 * count + 7) / 8;
    default:
      return 0;
  }
}

// Features of a token the per-token kernels take (their grids count threads
// in 32 bits).
constexpr int64_t kMaxFeatures = INT64_C(1) << 26;

inline bool is_float_io(thl_dtype t) { return t == THL_F32 || t == THL_F16 || t == THL_BF16; }

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi), empty when lo == hi
};

// Byte range spanned by a column-major r x c matrix with leading dimension ld.
inline Range matrix_range(const void* p, thl_dtype t, int64_t r, int64_t c, int64_t ld) {
  Range g;
  if (!p || r <= 0 || c <= 0) return g;
  g.lo = reinterpret_cast<uintptr_t>(p);
  g.hi = g.lo + static_cast<uintptr_t>(bytes_of(t, (c - 1) * ld + r));
  return g;
}

// Byte range of a device vector of `count` elements of `size` bytes.
inline Range vector_range(const void* p, int64_t count, int64_t size) {
  Range g;
  if (!p || count <= 0) return g;
  g.lo = reinterpret_cast<uintptr_t>(p);
  g.hi = g.lo + static_cast<uintptr_t>(count) * static_cast<uintptr_t>(size);
  return g;
}

inline bool overlaps(const Range& a, const Range& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

}  // namespace thl

// Host-side argument checks shared by the C ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

inline size_t io_bytes(int dtype) { return dtype == GDN_F16 ? 2 : 4; }

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
  Span() = default;
  Span(const void* p, size_t bytes) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + (p ? bytes : 0)) {}
  bool empty() const { return lo == hi; }
  bool overlaps(const Span& o) const { return !empty() && !o.empty() && lo < o.hi && o.lo < hi; }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cu[0] = 0 <= cu[1] <= ... <= cu[R] = N.
inline bool cu_host_ok(const int32_t* cu, int64_t R, int64_t N) {
  if (cu[0] != 0) return false;
  for (int64_t r = 0; r < R; ++r)
    if (cu[r + 1] < cu[r]) return false;
  return cu[R] == N;
}

}  // namespace gdn

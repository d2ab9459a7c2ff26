// The search for the K-th highest of a list's scores: which keys are taken, and how many of those that are equal to the
// last. Plain C++ without a device's functions, so that the kernels' own arithmetic also runs on the host.
#pragma once

#include <stdint.h>

namespace gdn {

#define GDN_INLINE __attribute__((always_inline)) constexpr

// Scores are kept as 64-bit keys that order as they do: 0 for an entry that may not be
// selected, one below the highest for a NaN, the highest for an entry that is always in.
constexpr uint64_t kAlways = ~(uint64_t)0;
GDN_INLINE uint64_t key_of(double x) {
  if (x != x) return kAlways - 1;
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  return (b >> 63) != 0 ? ~b : b | ((uint64_t)1 << 63);
}

struct Three {
  int a, b, c;
};

// Narrows [lo, hi], with `count` keys from lo on, K or more, and fewer than K above hi, until count is K or lo is hi;
// counts(x, y, z) says how many keys there are from each of the cuts x >= y >= z on (two ways: from y).
template <int WAYS, typename T, typename Counts>
GDN_INLINE void cut_range(int K, int& count, T& lo, T& hi, Counts counts) {
  while (count != K && lo < hi) {
    const T range = hi - lo, part = range >> 2;            // lo < z <= y <= x <= hi
    const T y = hi - (range >> 1), x = WAYS == 2 || range < 4 ? y : hi - part, z = WAYS == 2 || range < 4 ? y : y - part;
    const Three n = counts(x, y, z);
    if (WAYS == 4 && n.a >= K) {
      lo = x;
      count = n.a;
    } else if (n.b >= K) {
      lo = y;
      count = n.b;
      if (WAYS == 4) hi = x - 1;
    } else if (WAYS == 4 && n.c >= K) {
      lo = z;
      count = n.c;
      hi = y - 1;
    } else {
      hi = z - 1;
    }
  }
}

// A key's place in the range from lo on, in 32 bits: what is always in is above every cut, what is none below.
struct ShortKeys {
  uint64_t lo;
  int shift;
  GDN_INLINE uint32_t of(uint64_t key) const { return key == kAlways ? ~0u : key < lo ? 0 : (uint32_t)((key - lo) >> shift); }
};

// Keys from `least` on are taken, but for the last `surplus` of those that are equal to it.
struct Cut {
  uint64_t least;
  int surplus;
};

// The cut that leaves K of a list's `there` keys, K at most of which are kAlways; [lo, hi] holds all others. First by
// the 32 highest bits of the range, where a comparison takes a quarter of the time, then, where these do not tell the
// K-th from the next, by all: short_counts and counts are cut_range's of the short keys, which prepare(ShortKeys)
// announces, and of the keys.
template <int WAYS, typename Prepare, typename ShortCounts, typename Counts>
GDN_INLINE Cut find_cut(int K, int there, uint64_t lo, uint64_t hi, Prepare prepare, ShortCounts short_counts, Counts counts) {
  int count = there;                                       // from lo on there are K or more, above hi fewer
  const uint64_t range = hi - lo;
  if (range > 0) {
    const int bits = 64 - __builtin_clzll(range), shift = bits > 32 ? bits - 32 : 0;
    uint32_t lo32 = 0, hi32 = (uint32_t)(range >> shift);
    prepare(ShortKeys{lo, shift});
    cut_range<WAYS>(K, count, lo32, hi32, short_counts);
    // the last key that hi32 stands for, as a distance from lo: a NaN's key plus what its low bits leave out passes 2^64
    const uint64_t past = (uint64_t)hi32 << shift | (((uint64_t)1 << shift) - 1);
    hi = lo + (range < past ? range : past);
    lo += (uint64_t)lo32 << shift;
  }
  cut_range<WAYS>(K, count, lo, hi, counts);
  return Cut{lo, count - K};
}

#undef GDN_INLINE

}  // namespace gdn

// Selection of the pages that a token attends: gdn_kv_bounds and gdn_attn_select.
//
// A page's keys lie channel by channel within [low, high], so q . k over the page is at
// most sum_d max(q_d low_d, q_d high_d): for the heads that share a key head, w+ . high +
// w- . low with w+ (w-) the group's sum of the positive (negative) parts of q. That is two
// rows of D elements a page and head instead of page_size rows: the pages of the highest
// bounds are selected.
//
// Both are bound by the latency of lengths -> table -> keys or bounds, and the selection by its 64-bit sums too.
// Measured: bounds of 64 new tokens, 8 key heads of 128 fp16, pages of 64, 3.7 us (a launch); of prompts of 28,746 tokens,
// 4 of 256 in 8 bits, 31 MB, 10.5 us. Selection for 64 requests x 8 key heads, 32 of up to 256 pages, 30 MB, 13.6 us
// (about 11 the scores, 3 the list); 3 drafts x 4 key heads of 256 fp32, 128 of 4,097 pages, 34 MB, 25.6 us.
#include <type_traits>

#include "gdn_attn_kernels.h"
#include "gdn_common.h"
#include "gdn_pick.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// A launch takes fewer than 2^32 work-items in a dimension (more are dropped without an error), of workgroups of up to
// 1,024: they walk what is left.
constexpr int64_t kMostBlocks = (int64_t)1 << 21;

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

// Request that token n < the requests' tokens belongs to, found by a whole wave.
__device__ __forceinline__ int owner_of(const RowArgs& p, int n, int lane) {
  if (p.cu_seqlens == nullptr) return min((int)((unsigned)n / (unsigned)p.dense_len), p.R - 1);
  int owner = 0;
  for (int first = 0; first < p.R; first += 64) {
    const int i = first + lane;
    const int ended = __builtin_popcountll(__ballot(i < p.R && row_start(p, min(i, p.R - 1) + 1) <= n));
    owner += ended;
    if (ended < 64) break;
  }
  return __builtin_amdgcn_readfirstlane(min(owner, p.R - 1));
}

// ---------------------------------------------------------------------------- bounds

// The lower (higher) of two, NaN where one is.
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
template <typename IO> __device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b);
template <typename IO> __device__ __forceinline__ uint32_t higher(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t lower<_Float16>(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_minimum(__builtin_bit_cast(half2_t, a), __builtin_bit_cast(half2_t, b)));
}
template <> __device__ __forceinline__ uint32_t higher<_Float16>(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_maximum(__builtin_bit_cast(half2_t, a), __builtin_bit_cast(half2_t, b)));
}
template <> __device__ __forceinline__ uint32_t lower<float>(uint32_t a, uint32_t b) {
  return __float_as_uint(__builtin_elementwise_minimum(__uint_as_float(a), __uint_as_float(b)));
}
template <> __device__ __forceinline__ uint32_t higher<float>(uint32_t a, uint32_t b) {
  return __float_as_uint(__builtin_elementwise_maximum(__uint_as_float(a), __uint_as_float(b)));
}

// What a lane of the bounds kernel holds of a key: 16 bytes of the cache, as kWords dwords of io values. (8- and 4-bit
// elements are rounded to io before they are compared, which keeps their order.)
template <typename IO, int FMT>
struct Piece {
  static constexpr int kChannels = FMT == kCacheIo ? 16 / sizeof(IO) : FMT == kCacheE4M3 ? 16 : 32;
  static constexpr int kWords = kChannels * sizeof(IO) / 4;
};
template <typename IO, int FMT>
__device__ __forceinline__ void unpack(uint4_t raw, int s, uint32_t (&w)[Piece<IO, FMT>::kWords]) {
  const float scale = __uint_as_float((uint32_t)s << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == kCacheIo) {
      w[i] = raw[i];
    } else if constexpr (FMT == kCacheE4M3) {
      w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[i], scale, false));
      w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[i], scale, true));
    } else {
      w[4 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(raw[i], scale, 0));
      w[4 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(raw[i], scale, 1));
      w[4 * i + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(raw[i], scale, 2));
      w[4 * i + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(raw[i], scale, 3));
    }
  }
}

// f over the lanes whose numbers differ in the bits from E on (2 .. 32), without the LDS crossbar.
template <int E, typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F f) {
  const auto moved = [](uint32_t v, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, true);
  };
  if constexpr (E <= 2) x = f(x, moved(x, std::integral_constant<int, kDppQuadXor2>()));
  if constexpr (E <= 4)                                    // 7 - i, then 3 - i within 4: i ^ 4
    x = f(x, moved(moved(x, std::integral_constant<int, kDppHalfMirror>()), std::integral_constant<int, 0x1B>()));
  if constexpr (E <= 8) x = f(x, moved(x, std::integral_constant<int, 0x128>()));   // row_ror 8: i ^ 8
  if constexpr (E <= 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f(a[0], a[1]);
  }
  if constexpr (E <= 32) {
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = f(b[0], b[1]);
  }
  return x;
}

// The pages that hold the new tokens of request r: entries [first, first + count) of its table.
struct Touched {
  int first, count, len;
};
__device__ __forceinline__ Touched touched_of(const BoundsArgs& p, int r) {
  const int T = max(row_start(p.rows, r + 1) - row_start(p.rows, r), 0);
  const int64_t cap = (int64_t)p.cache.max_pages << p.cache.page_shift, len = p.rows.seq_lens[r];
  // positions [len - T, len) that the table holds
  const int64_t lo = min(max(len - T, (int64_t)0), cap), hi = min(max(len, (int64_t)0), cap);
  Touched x;
  x.first = (int)(lo >> p.cache.page_shift);
  x.count = hi > lo ? (int)((hi - 1) >> p.cache.page_shift) - x.first + 1 : 0;
  x.len = (int)hi;
  return x;
}

// The slot-th page of all requests' pages, laid end to end, found by a whole wave; r = -1 where there are fewer.
struct Slot {
  int r, entry, len;
};
__device__ __forceinline__ Slot slot_at(const BoundsArgs& p, int slot, int lane) {
  const int R = p.rows.R, per = (R + 63) >> 6, r0 = min(lane * per, R), r1 = min(r0 + per, R);
  int mine = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) mine += touched_of(p, r).count;
  int after = mine;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int y = __shfl_up(after, m);
    if (lane >= m) after += y;
  }
  Slot x{-1, 0, 0};
  const uint64_t holds = __ballot(slot >= after - mine && slot < after);
  if (holds == 0) return x;
  const int holder = __builtin_ctzll(holds);
  int left = slot - __builtin_amdgcn_readlane(after - mine, holder);
  for (int r = holder * per; r < R; ++r) {
    const Touched t = touched_of(p, r);
    if (left < t.count) {
      x = Slot{r, t.first + left, t.len};
      break;
    }
    left -= t.count;
  }
  return x;
}

// WAVES waves (a workgroup, or each of its 4) a page and head. kAhead keys of a lane's are on their way at once, so that
// most pages cost one wait.
constexpr int kAheadKeys = 4;
template <typename IO, int D, int FMT, int WAVES>
__global__ void __launch_bounds__(kThreads) gdn_kv_bounds_k(BoundsArgs p) {
  typedef Piece<IO, FMT> P;
  constexpr int E = D / P::kChannels;                      // lanes of a key
  constexpr int kAtOnce = 64 * WAVES / E, kAhead = kAheadKeys, W = P::kWords, kRow = D * (int)sizeof(IO) / 4;
  __shared__ uint32_t ends[WAVES > 1 ? WAVES : 1][2][WAVES > 1 ? kRow : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int tid = WAVES > 1 ? (int)threadIdx.x : lane, e = tid % E;
  const unsigned jobs = (unsigned)p.slots * (unsigned)p.cache.Hk, step = WAVES > 1 ? gridDim.x : gridDim.x * kWaves;
  for (unsigned job = WAVES > 1 ? blockIdx.x : blockIdx.x * kWaves + wave; job < jobs; job += step) {
    const unsigned slot = job / (unsigned)p.cache.Hk;      // 64-bit divisions would take a microsecond
    const int h = (int)(job - slot * p.cache.Hk);
    const Slot x = slot_at(p, (int)slot, lane);
    if (x.r < 0) return;
    const int64_t first = (int64_t)x.entry << p.cache.page_shift, row = cache_row(p.cache, x.r, first);
    if (row < 0) continue;                                 // uniform
    const int64_t row0 = row + ((int64_t)h << p.cache.page_shift);
    const int count = min(1 << p.cache.page_shift, x.len - (int)first);
    const char* keys = static_cast<const char*>(p.cache.k) + row0 * (16 * E) + 16 * e;
    const uint8_t* scales = FMT == kCacheE2M1 ? p.cache.k_scales + block_scale_at(row0, e, p.cache.page_shift, D)
                                              : p.cache.k_scales + row0;
    uint32_t lo[W], hi[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      lo[i] = sizeof(IO) == 2 ? 0x7c007c00u : 0x7f800000u; // infinities
      hi[i] = sizeof(IO) == 2 ? 0xfc00fc00u : 0xff800000u;
    }
    for (int k0 = tid / E; k0 < count; k0 += kAhead * kAtOnce) {
      uint4_t raw[kAhead];
      int s[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = min(k0 + u * kAtOnce, count - 1);    // past the last the last again
        raw[u] = *reinterpret_cast<const uint4_t*>(keys + (int64_t)k * (16 * E));
        s[u] = FMT == kCacheIo ? 0 : scales[k];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        uint32_t w[W];
        unpack<IO, FMT>(raw[u], s[u], w);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          lo[i] = lower<IO>(lo[i], w[i]);
          hi[i] = higher<IO>(hi[i], w[i]);
        }
      }
    }
    // over the lanes that hold the same channels: those E, 2 E .. apart
#pragma unroll
    for (int i = 0; i < W; ++i) {
      lo[i] = over_lanes<E>(lo[i], [](uint32_t a, uint32_t b) { return lower<IO>(a, b); });
      hi[i] = over_lanes<E>(hi[i], [](uint32_t a, uint32_t b) { return higher<IO>(a, b); });
    }
    uint32_t* out = static_cast<uint32_t*>(p.bounds) + (row0 >> p.cache.page_shift) * 2 * kRow;
    if (lane < E) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        (WAVES > 1 ? ends[wave][0] : out)[W * e + i] = lo[i];
        (WAVES > 1 ? ends[wave][1] : out + kRow)[W * e + i] = hi[i];
      }
    }
    if constexpr (WAVES == 1) continue;
    __syncthreads();
    for (int i = tid; i < 2 * kRow; i += kThreads) {
      const int high = i >= kRow ? 1 : 0, at = i - high * kRow;
      uint32_t m = ends[0][high][at];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) m = high ? higher<IO>(m, ends[w][high][at]) : lower<IO>(m, ends[w][high][at]);
      out[i] = m;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------- selection

template <int CTRL>
__device__ __forceinline__ double dpp64(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// Token n of request r: the request's table, the entries of it that the token holds.
struct Token {
  const int32_t* table;
  int64_t pos;
  int held;
};
__device__ __forceinline__ int held_at(const SelectArgs& p, int64_t pos) {
  return pos < 0 ? 0 : (int)min((pos >> p.cache.page_shift) + 1, (int64_t)p.cache.max_pages);
}
__device__ __forceinline__ Token token_at(const SelectArgs& p, int r, int n) {
  Token t;
  t.pos = (int64_t)p.rows.seq_lens[r] - row_start(p.rows, r + 1) + n;
  t.table = p.cache.table + (int64_t)r * p.cache.max_pages;
  t.held = held_at(p, t.pos);
  return t;
}

// 16 bytes of io elements as they are, and as doubles.
template <typename IO> struct Vec;
template <> struct Vec<_Float16> {
  typedef half8_t type;
};
template <> struct Vec<float> {
  typedef float4_t type;
};

// The group's sums of the negative and of the positive parts of q, channel by channel, each channel by one thread, for
// `count` tokens from n on.
template <typename IO, int D, int TOKENS>
__device__ __forceinline__ void sum_parts(const SelectArgs& p, int n, int count, int h, double (&parts)[TOKENS][2][D]) {
  const int d = threadIdx.x;
  if (d >= D) return;
  const IO* q = static_cast<const IO*>(p.q) + (int64_t)n * p.q_stride + (int64_t)h * p.group * D + d;
  double minus[TOKENS], plus[TOKENS];
#pragma unroll
  for (int j = 0; j < TOKENS; ++j) minus[j] = plus[j] = 0.0;
#pragma unroll 4
  for (int g = 0; g < p.group; ++g) {
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const float x = (float)q[min(j, count - 1) * p.q_stride + (int64_t)g * D];
      minus[j] += (double)(x > 0.f ? 0.f : x);             // a NaN goes into both
      plus[j] += (double)(x < 0.f ? 0.f : x);
    }
  }
#pragma unroll
  for (int j = 0; j < TOKENS; ++j) {
    parts[j][0][d] = minus[j];
    parts[j][1][d] = plus[j];
  }
}

// Scores of the entries [i0, i1) of a table, for the tokens whose parts are in LDS: L lanes an entry, 16 channels of both
// bounds each; kAhead entries of a lane's are on their way at once (a list of 256 entries took 18 us one at a time).
template <typename IO, int D>
struct Scorer {
  static constexpr int L = D / 16, V = 16 / sizeof(IO), kVecs = 16 / V, kAhead = 4, kStep = kThreads / L;
  typedef typename Vec<IO>::type vec_t;
  const SelectArgs& p;
  const int32_t* table;
  int h, i, i1;                                            // this lane's next entry, the end
  int page[kAhead], next[kAhead];
  uint4_t lo[kAhead][kVecs], hi[kAhead][kVecs];
  double minus[16], plus[16];

  __device__ __forceinline__ Scorer(const SelectArgs& args, const int32_t* entries, int head, int begin, int end)
      : p(args), table(entries), h(head), i(begin + (int)threadIdx.x / L), i1(end) {
    look_up();
  }
  __device__ __forceinline__ void look_up() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = table[min(i + u * kStep, i1 - 1)];
  }
  __device__ __forceinline__ void load() {
    const int e = threadIdx.x % L;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      page[u] = next[u] >= 0 && next[u] < p.cache.num_pages ? next[u] : -1;
      const IO* low = static_cast<const IO*>(p.bounds) + ((int64_t)max(page[u], 0) * p.cache.Hk + h) * 2 * D;
#pragma unroll
      for (int c = 0; c < kVecs; ++c) {
        lo[u][c] = *reinterpret_cast<const uint4_t*>(low + V * (c * L + e));
        hi[u][c] = *reinterpret_cast<const uint4_t*>(low + D + V * (c * L + e));
      }
    }
  }
  // Keeps the compiler from holding the bounds as doubles from token to token, in four times the registers.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int c = 0; c < kVecs; ++c) asm volatile("" : "+v"(lo[u][c]), "+v"(hi[u][c]));
  }
  __device__ __forceinline__ void take(const double (&parts)[2][D]) {
    const int e = threadIdx.x % L;
#pragma unroll
    for (int c = 0; c < kVecs; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        minus[V * c + k] = parts[0][V * (c * L + e) + k];
        plus[V * c + k] = parts[1][V * (c * L + e) + k];
      }
  }
  // store(entry, page, score) for the loaded entries and the token that was taken, by an entry's first lane.
  template <typename Store>
  __device__ __forceinline__ void score(Store store) const {
    const int e = threadIdx.x % L;
    double sum[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) sum[u] = 0.0;
#pragma unroll
    for (int c = 0; c < kVecs; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          sum[u] = fma(plus[V * c + k], (double)(float)__builtin_bit_cast(vec_t, hi[u][c])[k],
                       fma(minus[V * c + k], (double)(float)__builtin_bit_cast(vec_t, lo[u][c])[k], sum[u]));
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      double x = sum[u];
      x += dpp64<kDppQuadXor1>(x);
      x += dpp64<kDppQuadXor2>(x);
      if constexpr (L >= 8) x += dpp64<kDppHalfMirror>(x);
      if constexpr (L >= 16) x += dpp64<kDppRowMirror>(x);
      const int at = i + u * kStep;
      if (e == 0 && at < i1) store(at, page[u], x);
    }
  }
  // On to the next entries; false where there are none for any lane of the workgroup.
  __device__ __forceinline__ bool advance() {
    i += kAhead * kStep;
    if (i - (int)threadIdx.x / L >= i1) return false;
    look_up();
    load();
    return true;
  }
};

// The key of an entry of a token that holds `held`.
__device__ __forceinline__ uint64_t entry_key(const SelectArgs& p, int held, int at, int page, double score) {
  return page < 0 ? 0 : at < p.first || at >= held - p.newest ? kAlways : key_of(score);
}

// Writes the list's tail and its length.
template <int WAVES>
__device__ __forceinline__ void end_list(const SelectArgs& p, int count, int32_t* list, int32_t* count_out) {
  for (int i = count + (int)threadIdx.x; i < p.K; i += 64 * WAVES) list[i] = -1;
  if (threadIdx.x == 0 && count_out != nullptr) *count_out = count;
}

__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(x >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
}
// Largest over a wave's lanes.
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_max(uint64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, 0xF, 0xF, true);
  return max(x, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint64_t lane_of(uint64_t x, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
  x = dpp_max<kDppRowMirror>(dpp_max<kDppHalfMirror>(dpp_max<kDppQuadXor2>(dpp_max<kDppQuadXor1>(x))));
  return max(max(lane_of(x, 0), lane_of(x, 16)), max(lane_of(x, 32), lane_of(x, 48)));
}
// Sum over aligned groups of 16 lanes.
__device__ __forceinline__ int row_sum(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, kDppQuadXor1, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, kDppQuadXor2, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, kDppHalfMirror, 0xF, 0xF, true);
  return x + __builtin_amdgcn_update_dpp(0, x, kDppRowMirror, 0xF, 0xF, true);
}
__device__ __forceinline__ int count_lanes(bool x) { return __builtin_popcountll(__ballot(x)); }

// What the waves of a workgroup that share a list's keys tell each other. `turn` alternates, so that one barrier is enough.
struct PickShared {
  uint64_t low[16], high[16];
  int counts[2][4][16];
};

// The K entries of the highest keys among `held`, equal ones from the lowest entry on, in ascending order. A
// threshold is found by cutting the keys' range into WAYS parts until K keys lie from it on, or none but equal ones are
// left between its ends: as often as it takes to tell the K-th key from the next, 12 to 15 halvings among some
// thousand scores, 64 at most. Nothing is written outside the list's K places, whatever the keys.
//
// SHARED: the keys are split over the workgroup's waves, up to COLUMNS columns of 64 neighbours each (COLUMNS 0: any
// number, read again each time), which add their counts behind a barrier; else WAVES is 1.
constexpr int kColumns = 8, kFew = 64 * kColumns;          // keys that a wave holds in registers
template <int WAVES, int COLUMNS, bool SHARED, typename Keys>
__device__ __forceinline__ void pick(const SelectArgs& p, const Keys& keys, int held, int32_t* list, int32_t* count_out,
                                     PickShared& s) {
  constexpr int WAYS = SHARED ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int columns = (held + (SHARED ? 64 * WAVES : 64) - 1) / (SHARED ? 64 * WAVES : 64);
  const int first = SHARED ? wave * columns : 0;           // column of this wave
  uint64_t mine[COLUMNS > 0 ? COLUMNS : 1];
  const auto load = [&](int c) -> uint64_t {
    const int64_t i = 64 * (int64_t)(first + c) + lane;
    return i < held ? keys[i] : 0;
  };
  // f(key, column) of this wave's keys, all lanes together
  const auto each = [&](auto f) {
    if constexpr (COLUMNS > 0) {
#pragma unroll
      for (int c = 0; c < COLUMNS; ++c)
        if (c < columns) f(mine[c], c);
    } else {
      for (int c = 0; c < columns; ++c) f(load(c), c);
    }
  };
  if constexpr (COLUMNS > 0) {
#pragma unroll
    for (int c = 0; c < COLUMNS; ++c) mine[c] = c < columns ? load(c) : 0;
  }
  int turn = 0;
  // Sums over the waves of three numbers: row i of 16 lanes adds the waves' i-th. One read of LDS a wave (each wave
  // reading all of them took most of the time), and no array of the numbers, which the compiler would put into LDS by
  // the thread's number, read from the launch's packet in host memory (512 workgroups: 13 us).
  const auto total = [&](int a, int b, int c) -> Three {
    if constexpr (!SHARED) return Three{a, b, c};
    if (lane < 3) s.counts[turn][lane][wave] = lane == 0 ? a : lane == 1 ? b : c;
    __syncthreads();
    const int x = row_sum((lane & 15) < WAVES ? s.counts[turn][lane >> 4][lane & 15] : 0);
    turn ^= 1;
    return Three{__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16), __builtin_amdgcn_readlane(x, 32)};
  };

  uint64_t hi = 0, lo = kAlways;
  int some = 0, always = 0;
  each([&](uint64_t key, int) {
    some += count_lanes(key != 0);
    always += count_lanes(key == kAlways);
    hi = key != kAlways ? max(hi, key) : hi;
    lo = key != 0 ? min(lo, key) : lo;
  });
  const Three have = total(some, always, 0);
  const int there = have.a;
  uint64_t least = 1;                                      // keys from this one on are taken, but for the last
  int surplus = 0;                                         // of those that are equal to it
  if (there > p.K && have.b == p.K) {
    least = kAlways;
  } else if (there > p.K) {
    lo = ~wave_max(~lo);
    hi = wave_max(hi);
    if constexpr (SHARED) {
      if (lane == 0) {
        s.low[wave] = lo;
        s.high[wave] = hi;
      }
      __syncthreads();
      lo = ~wave_max(lane < WAVES ? ~s.low[lane] : 0);
      hi = wave_max(lane < WAVES ? s.high[lane] : 0);
    }
    uint32_t short_keys[COLUMNS > 0 ? COLUMNS : 1];
    ShortKeys shorts{0, 0};
    const auto prepare = [&](ShortKeys x) {
      shorts = x;
      if constexpr (COLUMNS > 0) {
#pragma unroll
        for (int c = 0; c < COLUMNS; ++c) {
          short_keys[c] = c < columns ? shorts.of(mine[c]) : 0;
          asm("" : "+v"(short_keys[c]));                   // a number from here on: else each cut asks again what is always in
        }
      }
    };
    const auto short_counts = [&](uint32_t x, uint32_t y, uint32_t z) {
      int nx = 0, ny = 0, nz = 0;
      each([&](uint64_t key, int c) {
        const uint32_t k = COLUMNS > 0 ? short_keys[COLUMNS > 0 ? c : 0] : shorts.of(key);
        ny += count_lanes(k >= y);
        if constexpr (WAYS == 4) {
          nx += count_lanes(k >= x);
          nz += count_lanes(k >= z);
        }
      });
      return total(nx, ny, nz);
    };
    const Cut cut = find_cut<WAYS>(p.K, there, uniform(lo), uniform(hi), prepare, short_counts,
                                   [&](uint64_t x, uint64_t y, uint64_t z) {
      int nx = 0, ny = 0, nz = 0;
      each([&](uint64_t key, int) {
        ny += count_lanes(key >= y);
        if constexpr (WAYS == 4) {
          nx += count_lanes(key >= x);
          nz += count_lanes(key >= z);
        }
      });
      return total(nx, ny, nz);
    });
    least = cut.least;
    surplus = cut.surplus;
  }
  // before this wave's: what is taken, and how many of the keys equal to `least`
  int before = 0, kept = 0;
  if constexpr (SHARED) {
    int n = 0, equal = 0;
    each([&](uint64_t key, int) {
      n += count_lanes(key >= least);
      equal += count_lanes(key == least);
    });
    if (lane == 0) {
      s.counts[turn][0][wave] = n;
      s.counts[turn][1][wave] = equal;
    }
    __syncthreads();
    // rows of 16 lanes: what is taken before this wave, ties before it, all ties
    const int w = lane & 15, row = lane >> 4;
    const int x = row_sum(w < (row == 2 ? WAVES : wave) ? s.counts[turn][row == 0 ? 0 : 1][w] : 0);
    before = __builtin_amdgcn_readlane(x, 0);
    const int equal_before = __builtin_amdgcn_readlane(x, 16), all_equal = __builtin_amdgcn_readlane(x, 32);
    const int keep = all_equal - surplus;                  // of all ties, the first ones
    before -= max(equal_before - keep, 0);
    kept = max(keep - equal_before, 0);
  } else if (surplus > 0) {
    each([&](uint64_t key, int) { kept += count_lanes(key == least); });
    kept -= surplus;
  }
  const rsrc_t places = make_rsrc(list, 4 * p.K);          // whose bounds drop what lies outside
  int at = before;
  each([&](uint64_t key, int c) {
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    uint64_t in = __ballot(key >= least);
    if (surplus > 0) {
      const uint64_t ties = __ballot(key == least);
      in &= ~ties | __ballot(__builtin_popcountll(ties & below) < kept);
      kept -= __builtin_popcountll(ties);
    }
    if ((in >> lane & 1) != 0)
      __builtin_amdgcn_raw_buffer_store_b32((uint32_t)(64 * (first + c) + lane), places, 4 * (at + __builtin_popcountll(in & below)), 0, 0);
    at += __builtin_popcountll(in);
  });
  end_list<WAVES>(p, min(there, p.K), list, count_out);
}

extern __shared__ uint64_t lds_keys[];                     // p.lds_entries of them

// One list a workgroup: all of its keys, then the selection among them.
template <typename IO, int D>
__global__ void __launch_bounds__(kThreads) gdn_attn_select_k(SelectArgs p) {
  __shared__ PickShared shared;
  __shared__ double parts[1][2][D];
  const unsigned lists = (unsigned)min(row_start(p.rows, p.rows.R), p.rows.N) * (unsigned)p.cache.Hk;
  for (unsigned job = blockIdx.x; job < lists; job += gridDim.x) {
    const int n = (int)(job / (unsigned)p.cache.Hk), h = (int)job - n * p.cache.Hk;
    const Token t = token_at(p, owner_of(p.rows, n, threadIdx.x & 63), n);
    int32_t *list = p.pages + (int64_t)job * p.K, *count = h == 0 ? p.counts + n : nullptr;
    uint64_t* keys = p.keys + (int64_t)job * p.cache.max_pages;
    const bool in_lds = t.held <= p.lds_entries;
    if (t.held > 0) {
      sum_parts<IO, D, 1>(p, n, 1, h, parts);
      Scorer<IO, D> s(p, t.table, h, 0, t.held);
      __syncthreads();
      s.take(parts[0]);
      s.load();
      do {
        s.score([&](int at, int page, double x) { (in_lds ? lds_keys[at] : keys[at]) = entry_key(p, t.held, at, page, x); });
      } while (s.advance());
      __syncthreads();
    }
    if (!in_lds)
      pick<kWaves, 0, true>(p, keys, t.held, list, count, shared);
    else if (threadIdx.x < 64)
      pick<1, kColumns, false>(p, lds_keys, t.held, list, count, shared);
    __syncthreads();
  }
}

// Long lists in two launches: the keys of p.chunk entries for TOKENS tokens a workgroup (those of one request
// share the bounds that they read), then the selection.
template <typename IO, int D, int TOKENS>
__global__ void __launch_bounds__(kThreads) gdn_select_score_k(SelectArgs p) {
  __shared__ double parts[TOKENS][2][D];
  const int tokens = min(row_start(p.rows, p.rows.R), p.rows.N);
  const unsigned jobs = ((unsigned)p.rows.N + TOKENS - 1) / TOKENS * (unsigned)p.cache.Hk;
  for (unsigned job = blockIdx.x; job < jobs; job += gridDim.x) {
    const unsigned group = job / (unsigned)p.cache.Hk;
    const int h = (int)(job - group * p.cache.Hk), past = min((int)group * TOKENS + TOKENS, tokens);
    int n = (int)group * TOKENS;
    while (n < past) {
      // the tokens from n on that are of one request: the last of them holds the most entries
      const int r = owner_of(p.rows, n, threadIdx.x & 63);
      const int count = max(min(past, row_start(p.rows, r + 1)) - n, 1);   // on, whatever cu_seqlens holds
      const Token t = token_at(p, r, n + count - 1);
      // the last chunk takes what the host did not know of
      const int i0 = min((int)blockIdx.y * p.chunk, t.held);
      const int i1 = blockIdx.y == gridDim.y - 1 ? t.held : min(i0 + p.chunk, t.held);
      if (i0 < i1) {
        Scorer<IO, D> s(p, t.table, h, i0, i1);
        s.load();
        sum_parts<IO, D, TOKENS>(p, n, count, h, parts);
        __syncthreads();
        if (TOKENS == 1) s.take(parts[0]);
        do {
#pragma unroll 1
          for (int j = 0; j < (TOKENS == 1 ? 1 : count); ++j) {
            if (TOKENS > 1) {
              s.forget();
              s.take(parts[j]);
            }
            const int held = held_at(p, t.pos - (count - 1 - j));
            uint64_t* keys = p.keys + ((int64_t)(n + j) * p.cache.Hk + h) * p.cache.max_pages;
            s.score([&](int at, int page, double x) {
              if (at < held) keys[at] = entry_key(p, held, at, page, x);
            });
          }
        } while (s.advance());
        __syncthreads();                                   // parts are written again
      }
      n += count;
    }
  }
}

template <int WAVES>
__global__ void __launch_bounds__(64 * WAVES) gdn_select_pick_k(SelectArgs p) {
  __shared__ PickShared shared;
  const unsigned lists = (unsigned)min(row_start(p.rows, p.rows.R), p.rows.N) * (unsigned)p.cache.Hk;
  for (unsigned job = blockIdx.x; job < lists; job += gridDim.x) {
    const int n = (int)(job / (unsigned)p.cache.Hk);
    const Token t = token_at(p, owner_of(p.rows, n, threadIdx.x & 63), n);
    int32_t *list = p.pages + (int64_t)job * p.K, *count = (int)job == n * p.cache.Hk ? p.counts + n : nullptr;
    const uint64_t* keys = p.keys + (int64_t)job * p.cache.max_pages;
    if (t.held > kFew * WAVES)
      pick<WAVES, 0, true>(p, keys, t.held, list, count, shared);
    else if (WAVES > 1 && t.held > kFew)
      pick<WAVES, kColumns, true>(p, keys, t.held, list, count, shared);
    else if (threadIdx.x < 64)
      pick<1, kColumns, false>(p, keys, t.held, list, count, shared);
    __syncthreads();
  }
}

unsigned blocks_of(int64_t jobs) { return (unsigned)(jobs < kMostBlocks ? jobs : kMostBlocks); }

// A wave a page where two rounds of its loads hold the page and the device is full anyway (28,746 tokens of 4 key heads
// of 256 in pages of 16, a wave against a workgroup: 4 bits 14 and 38 us, FP16 13 and 20).
template <typename IO, int D, int FMT>
hipError_t launch_bounds_f(const BoundsArgs& p, hipStream_t stream) {
  const int64_t jobs = (int64_t)p.slots * p.cache.Hk;
  constexpr int E = D / Piece<IO, FMT>::kChannels;
  if (jobs >= 1024 && (E << p.cache.page_shift) <= 2 * 64 * kAheadKeys)
    hipLaunchKernelGGL((gdn_kv_bounds_k<IO, D, FMT, 1>), dim3(blocks_of((jobs + kWaves - 1) / kWaves)), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((gdn_kv_bounds_k<IO, D, FMT, kWaves>), dim3(blocks_of(jobs)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <typename IO, int D>
hipError_t launch_bounds_d(const BoundsArgs& p, hipStream_t stream) {
  if constexpr (sizeof(IO) == 2) {
    if (p.cache.format == kCacheE4M3) return launch_bounds_f<IO, D, kCacheE4M3>(p, stream);
    if (p.cache.format == kCacheE2M1) return launch_bounds_f<IO, D, kCacheE2M1>(p, stream);
  }
  return p.cache.format == kCacheIo ? launch_bounds_f<IO, D, kCacheIo>(p, stream) : hipErrorInvalidValue;
}

template <typename IO>
hipError_t launch_bounds_io(const BoundsArgs& p, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_bounds_d<IO, 64>(p, stream);
    case 128: return launch_bounds_d<IO, 128>(p, stream);
    case 256: return launch_bounds_d<IO, 256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

// One launch where lists are short and few, so that their latency counts, two where they are split over workgroups or
// fill the device anyway. Measured, one against two, 8 key heads of 128 fp16 (bounds of 512 bytes): a request of 64
// pages 5.6 and 7.5 us, 64 of them 9.3 and 11.5, 256 of them 27.7 and 22.6; 64 of up to 256 pages 13.6 and 15.0; one
// of 2,048 37 and 12, 16 of 1,024 28 and 22. Between 256 and 512 pages few lists gain by two launches and many lose: of
// 300 pages one request 10.4 and 9.1, 4 10.6 and 9.5, 16 13.5 and 14.4, 64 20.0 and 23.5, 128 41 and 47; of 512 13.2 and
// 10.2, 13.3 and 10.6, 16.9 and 18.4, 32.3 and 39.5, 59 and 71. A length alone does not tell these apart; kShort is for
// the few.
constexpr int kShort = 256, kFewLists = 1024;
static_assert(kShort <= kFew, "a list in LDS is one wave's to pick from");

template <typename IO, int D>
hipError_t launch_select_d(SelectArgs p, hipStream_t stream) {
  const int64_t lists = (int64_t)p.rows.N * p.cache.Hk;
  if (p.max_held <= kShort && lists <= kFewLists) {
    p.lds_entries = p.max_held;
    hipLaunchKernelGGL((gdn_attn_select_k<IO, D>), dim3(blocks_of(lists)), dim3(kThreads), p.lds_entries * sizeof(uint64_t),
                       stream, p);
    return hipGetLastError();
  }
  // entries of a workgroup: 64 at least (what its lanes have on their way at once), about 1,024 workgroups
  const int64_t share = (lists * p.max_held / 1024 + 63) / 64 * 64, fits = (p.max_held + 32767) / 32768;
  p.chunk = (int)(share > 64 ? (share < (1 << 30) ? share : 1 << 30) : 64);
  if (p.chunk < fits) p.chunk = (int)fits;
  const int64_t jobs = ((int64_t)p.rows.N + p.group_tokens - 1) / p.group_tokens * p.cache.Hk;
  const dim3 grid(blocks_of(jobs), (unsigned)(p.max_held > 0 ? (p.max_held + p.chunk - 1) / p.chunk : 1));
  if (p.group_tokens == 1)
    hipLaunchKernelGGL((gdn_select_score_k<IO, D, 1>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((gdn_select_score_k<IO, D, kSelectGroup>), grid, dim3(kThreads), 0, stream, p);
  if (p.max_held <= kFew)
    hipLaunchKernelGGL(gdn_select_pick_k<1>, dim3(blocks_of(lists)), dim3(64), 0, stream, p);
  else if (p.max_held <= 4 * kFew)
    hipLaunchKernelGGL(gdn_select_pick_k<4>, dim3(blocks_of(lists)), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(gdn_select_pick_k<16>, dim3(blocks_of(lists)), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_select_io(const SelectArgs& p, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_select_d<IO, 64>(p, stream);
    case 128: return launch_select_d<IO, 128>(p, stream);
    case 256: return launch_select_d<IO, 256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_bounds(const BoundsArgs& p, int io_dtype, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  return io_dtype == 1 ? launch_bounds_io<_Float16>(p, stream) : launch_bounds_io<float>(p, stream);
}

hipError_t launch_select(const SelectArgs& p, int io_dtype, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  return io_dtype == 1 ? launch_select_io<_Float16>(p, stream) : launch_select_io<float>(p, stream);
}

}  // namespace gdn

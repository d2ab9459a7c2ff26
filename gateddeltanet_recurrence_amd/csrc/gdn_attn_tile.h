// Attention of every request's newest tokens over its paged cache: the kernels of
// gdn_attn_forward and gdn_attn_sparse_forward, instantiated by gdn_attn*.hip.
//
// With the scores x_t = scale log2(e) q.k_t of the attended positions, a row's
// output is sum_t 2^(x_t - M) v_t / sum_t 2^(x_t - M) for any M. A wave walks its
// positions once with a running M (the largest x so far, less a constant: kLift), l
// (the sum of the weights) and the output's unnormalised sum, rescaling both when M
// grows; waves, and workgroups that share a request's length, are joined by the same
// rule.
//
// Reading every key and value once for a few dozen rows (tokens x heads of a key
// head) is bound by HBM; the matrix cores keep the arithmetic out of the way. Rows
// are the N side of both products, S^T = K Q^T and O^T = V^T P^T: a row's scores
// lie in 4 lanes (l & 15 = row), its weights leave the first product in the order
// the second one takes them in, and the running M, l and the rescaling factor are
// one register each. Keys and values go straight from memory to registers, with no LDS
// and no barrier in the loop. A wave's tile is 32 positions (16 for fp32), the waves of
// a workgroup take alternate tiles, and each has 16 or 32 KiB of them in flight. Up to
// two tiles of 16 rows share the loaded keys and values.
//
// What this replaced: 8 waves fed from an LDS ring by two loader waves were slower
// wherever a segment has up to 32 rows (16 requests x 4 drafts x 6 heads a key head, up
// to 8,192 positions of D = 256 fp16: 74 us against 60) and for more rows, as several
// segments, in all but one case: 16 x 5 drafts x 8 heads over 4,096 positions, D = 256
// fp16 66 against 69, 8 bits 67 against 47, D = 64 fp16 37 against 25, D = 128 fp32
// 100 against 89 us.
//
// Work is split evenly over the workgroups whatever the lengths (short requests are not
// split at all, see one_group_each): the positions of every segment (request, 16 or 32
// rows, key head) in chunks of 128 are laid end to end, and workgroup b takes the b-th
// equal share of the chunks. A share that holds all of a segment's chunks writes the
// output; the others leave (M, l, sum) in the workspace and gdn_attn_join_k, a second
// launch, joins them. Every wave forms the prefix sums of the requests' chunks by
// itself: R loads and one scan instead of a launch. The order of every sum is fixed by
// the lengths, so results repeat bit for bit; no atomics are used.
//
// Measured: 64 requests of up to 16,384 positions, 8 key heads of 128 fp16, 1.85 GB, 294 us
// (6.3 TB/s; counted HBM reads equal the bytes of the attended keys and values); 16 x up
// to 4 drafts over up to 8,192 positions of 4 x 256 fp16, 279 MB, 60 us; one request of
// 131,072 positions in 8 bits, 270 MB, 51 us; one of 333 positions 8 us.
//
// 4-bit pages (GDN_CACHE_E2M1) have a scale per 32 elements, applied by the conversion to FP16, exactly: about 200 vector
// instructions for 32 positions of 128 columns, 64 of them conversions. More waves a SIMD hide more than more tiles in
// flight a wave do (see kMostAhead). 64 requests of up to 16,384, D = 128, 491 MB, 89 to 93 us (5.3 to 5.5 TB/s; its loop
// alone 6.4); 16 x up to 4 drafts over up to 8,191 positions, D = 256, 75 MB, 31.9 us, of which about 20 are the loop.
// Their M is the largest q.k itself: scale log2(e) and the lift are applied to a score's distance from it.
//
// LISTS: the positions of a token and key head are those of its listed pages, each list a segment of its own: 64 requests
// x 8 key heads x 32 pages of 64, D = 128 fp16, 530 MB, 86 to 90 us (5.9 to 6.2 TB/s, HBM); 2 drafts x 65 pages, D = 256
// in 4 bits, 13.6 us (latency, the join's 4 us among it).
#pragma once

#include <type_traits>

#include "gdn_attn_kernels.h"
#include "gdn_common.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;             // of gdn_attn_join_k
constexpr int kRows = 16;                 // rows of a tile: the N side of the MFMA
constexpr int kTiles = 2;                 // tiles of a segment, at most
constexpr int kChunkShift = 7;            // positions of a unit of work: 128 or more
constexpr int kMostLines = 8;             // see block_of
// Of segments that are not split, up to this many get a workgroup each. More are shared
// out over two a CU, which load a segment's first tiles before the last one is joined,
// evenly by length; a segment's fixed part counts as so many bytes of keys and values.
// One each against shared: 256 requests of 100 positions, 8 key heads of 128 fp16 43 and
// 34 us, of 300 70 and 62, of 90 .. 700 75 and 73; with 1,024 segments the uneven ones
// lose (128 requests of 1 .. 4 drafts, 64 columns in 8 bits, 28 and 32 us).
constexpr int kOneEach = 1024;
constexpr int kSegmentBytes = 200000;
constexpr int kSegmentBytes4 = 30000;     // of 4-bit pages: 256 of 90 .. 700, D = 128, 39.8 us, with 200,000 43.9
constexpr int64_t kMostShared = 1 << 22;
constexpr int64_t kMostUnits = (int64_t)1 << 30;   // of a launch: they are counted in 32 bits
constexpr int kWholeShift = 30;           // one unit per segment: nothing is split
constexpr int kGroups = 256;              // workgroups of a split launch: one per CU

enum Format { kF32 = 0, kF16 = 1, kE4M3 = 2, kE2M1 = 3 };

// The arguments of a launch over all positions, or over lists of pages.
template <bool LISTS> using Args = typename std::conditional<LISTS, SparseArgs, AttnArgs>::type;

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

struct SplitArgs {
  int4* notes;                            // of the segments that may be split (see note_segment); null: none is
  float* parts;                           // [2 * groups][part_rows * (D + 2)]: M, l, sums
  int32_t part_rows;
  int32_t seg_shift;                      // log2 of a segment's rows: 4 or 5
  int32_t line_shift, line_groups;        // log2 of the lines, workgroups of a line (see block_of)
  int32_t chunk_shift;                    // log2 of a unit's positions
  int32_t whole;                          // > 0: a share is the segments that begin in it
  int32_t more;                           // units that a segment's fixed part counts as: before its own where it is split
  int32_t max_segs;                       // > 0: notes by segment, this many of a request and key head; 0: by workgroup
};

// What a request brings: its rows, the positions any of them attends and its units.
struct Plan {
  int start, T;                           // first token, tokens
  int len;                                // seq_lens[r], 0 for less
  int base, hi;                           // positions [base, hi), base a multiple of 32
  int segs, chunks;                       // segments of a key head, units of each
};

// Tokens are at most 2^30 and lengths not negative here, so that their differences fit 32 bits.
__device__ __forceinline__ int clamp_pos(int x, int hi) { return min(max(x, 0), hi); }

// The first position that the token before `past` attends, at most hi.
__device__ __forceinline__ int window_start(const AttnArgs& p, int past, int hi) {
  return clamp_pos(__builtin_elementwise_sub_sat(past, p.window), hi);
}

// First token, tokens and length of request r. With lists a token is a request, as long as its list's pages.
struct RequestRow {
  int start, T, len;
};
template <bool LISTS>
__device__ __forceinline__ RequestRow row_of(const Args<LISTS>& p, int r) {
  RequestRow x;
  if constexpr (LISTS) {
    const int entries = p.counts != nullptr ? min(max(p.counts[r], 0), p.list_len) : p.list_len;
    x = RequestRow{r, r < row_start(p.owners, p.owners.R) ? 1 : 0, entries << p.cache.page_shift};
  } else {
    x.start = row_start(p.rows, r);
    x.T = max(row_start(p.rows, r + 1) - x.start, 0);
    x.len = p.rows.seq_lens[r];
  }
  return x;
}

// The positions that a table, or a list, holds.
template <bool LISTS>
__device__ __forceinline__ int capacity_of(const Args<LISTS>& p) {
  if constexpr (LISTS)
    return p.list_len << p.cache.page_shift;
  else
    return p.cache.max_pages << p.cache.page_shift;
}

template <bool LISTS>
__device__ __forceinline__ Plan plan_of(const Args<LISTS>& p, const SplitArgs& sp, int start, int T, int len) {
  Plan s;
  s.start = start;
  s.T = T;
  s.len = max(len, 0);
  const int cap = capacity_of<LISTS>(p);
  s.hi = min(s.len, cap);
  s.base = p.window > 0 ? window_start(p, s.len - s.T + 1, s.hi) & ~31 : 0;
  s.segs = (s.T * p.group + (1 << sp.seg_shift) - 1) >> sp.seg_shift;
  if (sp.max_segs > 0) s.segs = min(s.segs, sp.max_segs);  // no note past the request's, whatever cu_seqlens holds
  s.chunks = s.T > 0 ? max((int)(((unsigned)(s.hi - s.base) + (1u << sp.chunk_shift) - 1) >> sp.chunk_shift) + sp.more, 1) : 0;
  return s;
}

// The launch bounds the units of all requests by kMostUnits.
__device__ __forceinline__ int units_of(const SplitArgs& sp, const Plan& s, int Hk) {
  return (sp.line_shift > 0 ? 1 : s.segs) * Hk * s.chunks;
}

__device__ __forceinline__ int share_of(int total, int groups) {
  return total <= groups ? 1 : (int)((unsigned)(total + groups - 1) / (unsigned)groups);
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row 0's total to row 1, row 2's to row 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // the lower half's total to the upper
  return x;
}

struct Share {
  int u, u_end, r, r_first, size;
  int first, start, T, len;                                // of request first + lane
  int id, at, line;                                        // see block_of
};

// Where requests have 2 to 8 segments each, the same positions' segments go to as many
// workgroups (lines), which walk them at once and share an L2: workgroups are handed
// to the 8 XCDs in turn, so the numbers of those of one position differ by 8. `at` is a
// workgroup's place in its line, `id` its number line by line.
__device__ __forceinline__ void block_of(const SplitArgs& sp, Share& w) {
  const int b = (int)blockIdx.x;
  w.id = w.at = b;
  w.line = 0;
  if (sp.line_shift > 0) {
    const int slot = b >> 3;
    w.line = slot & ((1 << sp.line_shift) - 1);
    w.at = (slot >> sp.line_shift << 3) + (b & 7);
    w.id = w.line * sp.line_groups + w.at;
  }
}

// A request's plan: the lanes hold 64 of them, so that no load is in the way of the table's.
template <bool LISTS>
__device__ __forceinline__ Plan plan_at(const Args<LISTS>& p, const SplitArgs& sp, const Share& w, int r) {
  const int k = r - w.first;
  if (k < 64)
    return plan_of<LISTS>(p, sp, __builtin_amdgcn_readlane(w.start, k), __builtin_amdgcn_readlane(w.T, k),
                          __builtin_amdgcn_readlane(w.len, k));
  const RequestRow x = row_of<LISTS>(p, r);
  return plan_of<LISTS>(p, sp, x.start, x.T, x.len);
}

// This workgroup's share [u, u_end) of the units, and the request r that holds u,
// whose units begin at r_first. Every wave finds it by itself.
template <bool LISTS>
__device__ __forceinline__ Share find_share(const Args<LISTS>& p, const SplitArgs& sp, int lane) {
  const int R = p.rows.R, per = (R + 63) >> 6;             // requests a lane sums
  const int r0 = min(lane * per, R), r1 = min(r0 + per, R);
  int mine = 0;
  Share w;
  const auto hold = [&](int first) {
    const int r = min(first + lane, R - 1);
    const RequestRow x = row_of<LISTS>(p, r);
    w.first = first;
    w.start = x.start;
    w.T = x.T;
    w.len = x.len;
  };
  hold(0);
  if (R <= 64) {
    if (r0 < r1) mine = units_of(sp, plan_of<LISTS>(p, sp, w.start, w.T, w.len), p.cache.Hk);
  } else {
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      const RequestRow x = row_of<LISTS>(p, r);
      mine += units_of(sp, plan_of<LISTS>(p, sp, x.start, x.T, x.len), p.cache.Hk);
    }
  }
  const int after = wave_scan(mine), before = after - mine;
  const int total = __builtin_amdgcn_readlane(after, 63);
  block_of(sp, w);
  const int share = w.size = share_of(total, sp.line_groups);
  w.u = min(w.at * share, total);
  w.u_end = min(w.u + share, total);
  w.r = w.r_first = 0;
  if (w.u >= w.u_end) return w;
  const int holder = __builtin_ctzll(__ballot(w.u >= before && w.u < after));
  w.r = holder * per;
  w.r_first = __builtin_amdgcn_readlane(before, holder);
  if (R > 64) hold(w.r);
  if (sp.whole > 0) {
    // on to the first segment that begins here
    Plan s = plan_at<LISTS>(p, sp, w, w.r);
    while (w.u - w.r_first >= units_of(sp, s, p.cache.Hk)) {
      w.r_first += units_of(sp, s, p.cache.Hk);
      s = plan_at<LISTS>(p, sp, w, ++w.r);
    }
    const unsigned past = (unsigned)(w.u - w.r_first) % (unsigned)s.chunks;
    if (past > 0) w.u += s.chunks - (int)past;
  }
  return w;
}

// The token of a request that a row belongs to.
__device__ __forceinline__ int token_of(const AttnArgs& p, const Plan& s, int row) {
  return s.T == 1 ? 0 : p.group == 1 ? row : (int)((unsigned)row / (unsigned)p.group);
}

// The next segment of a share: units [c0, c1) of (request, rows from seg_row on, key
// head h); the share's u moves past it.
struct Segment {
  Plan s;
  int h, seg_row, rows, c0, c1;
  int t0, end;                                             // positions [t0, end)
  int id, note, last_unit;                                 // its workgroup, its place among the notes, its last unit
};

template <bool LISTS>
__device__ __forceinline__ Segment next_segment(const Args<LISTS>& p, const SplitArgs& sp, Share& w) {
  Segment x;
  x.s = plan_at<LISTS>(p, sp, w, w.r);
  while (w.u - w.r_first >= units_of(sp, x.s, p.cache.Hk)) {   // requests without tokens have no units
    w.r_first += units_of(sp, x.s, p.cache.Hk);
    x.s = plan_at<LISTS>(p, sp, w, ++w.r);
  }
  const unsigned local = w.u - w.r_first, seg = x.s.chunks == 1 ? local : local / (unsigned)x.s.chunks;
  x.c0 = local - seg * x.s.chunks;
  x.c1 = sp.whole > 0 ? x.s.chunks : min(x.s.chunks, x.c0 + (w.u_end - w.u));
  int line = w.line;
  x.h = seg;
  if (sp.line_shift == 0 && x.s.segs > 1) {
    x.h = seg / (unsigned)x.s.segs;
    line = seg - x.h * x.s.segs;
  }
  x.seg_row = line << sp.seg_shift;
  x.id = w.id;
  x.note = sp.max_segs > 0 ? (w.r * p.cache.Hk + x.h) * sp.max_segs + line : w.id;
  x.last_unit = w.u - x.c0 + x.s.chunks - 1;
  w.u += x.c1 - x.c0;
  x.rows = line < x.s.segs ? min(1 << sp.seg_shift, x.s.T * p.group - x.seg_row) : 0;   // 0: fewer segments than lines
  const int cap = capacity_of<LISTS>(p);
  const int past_last = x.rows == 0 ? 0 : x.s.len - x.s.T + token_of(p, x.s, x.seg_row + x.rows - 1) + 1;
  x.t0 = x.s.base + (max(x.c0 - sp.more, 0) << sp.chunk_shift);
  x.end = (int)min((unsigned)x.s.base + ((unsigned)(sp.whole > 0 ? x.c1 : max(x.c1 - sp.more, 0)) << sp.chunk_shift),
                   (unsigned)clamp_pos(past_last, cap));
  return x;
}

// The workgroup that begins a segment notes what the join has to know of it: the
// parts, the first of them, where the rows belong. In the order of workgroups there
// is one note each, of the last segment that it begins and leaves to others.
__device__ __forceinline__ void note_segment(const SplitArgs& sp, const Segment& x, const Share& w) {
  // the shares from this one on that hold the segment
  const int parts = x.c1 == x.s.chunks ? 0 : (int)((unsigned)x.last_unit / (unsigned)w.size) - w.at + 1;
  sp.notes[2 * x.note] = int4{parts, w.id, x.rows, x.seg_row};
  sp.notes[2 * x.note + 1] = int4{x.s.start, x.h, x.s.T, 0};
}

// Row n of a segment of `rows` rows from row0 on, and the positions that it attends:
// [lo, hi); every row of the segment attends [lo_max, hi_min).
struct Rows {
  int j, head;                                             // token of the request, head of the group
  int lo, hi, lo_max, hi_min;
};

template <bool LISTS>
__device__ __forceinline__ Rows rows_of(const Args<LISTS>& p, const Plan& s, int row0, int rows, int n) {
  Rows x;
  const int cap = capacity_of<LISTS>(p);
  const int last = row0 + max(rows, 1) - 1, row = min(row0 + n, min(last, s.T * p.group - 1));
  x.j = token_of(p, s, row);
  x.head = row - x.j * p.group;
  const int before = s.len - s.T + 1;                      // one past the first token's newest position
  const int past = before + x.j, past0 = before + token_of(p, s, row0), past1 = before + token_of(p, s, last);
  x.hi = n < rows ? clamp_pos(past, cap) : 0;
  x.hi_min = clamp_pos(past0, cap);
  x.lo = x.lo_max = 0;
  if (p.window > 0) {
    x.lo = window_start(p, past, cap);
    x.lo_max = window_start(p, past1, cap);
  }
  return x;
}

// Largest (sum) over the 4 lanes that hold a row: l & 15 the same.
__device__ __forceinline__ float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_maximum(float x) {     // NaN where one is
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __builtin_elementwise_maximum(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_elementwise_maximum(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Two e4m3 codes (the low or high half of a dword) as two fp16 values: exact.
template <bool HI>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// Two e2m1 codes (byte AT of a dword) times a power of two as two fp16 values: exact for the scales that a cache holds.
template <int AT>
__device__ __forceinline__ uint32_t nibbles_to_half2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, AT));
}

// The product with v takes fp16 operands. A weight w goes into it as two of them: hi, rounded toward zero, and
// lo = w - hi + 2^-11 hi, so that hi + lo is (1 + 2^-11) w to 2^-19 of it (or 2^-23, where fp16 ends), and the
// weights' sum takes the same factor. The share of hi in lo keeps lo from being 0 or negative, where an infinite
// value would become NaN. Rounded once to fp16, the weights made the output's error against 64 bits 6 to 11 % larger
// than its own rounding is. The second product and the split cost, one against two: 64 requests of up to 16,384
// positions 294.8 and 295.4 us, one of 333 8.3 and 8.4, a prompt of 300 tokens 21.3 and 22.2; with 8-bit pages, which
// wait for the vector units, one row tile 1 to 3 %, two 4 to 11 % (16 requests x 5 drafts x 8 heads over 4,096
// positions, D = 256, 48.1 and 52.1 us).
// Weights are also raised by 2^15, so that fp16's range below 1 is not all they have: a row keeps its digits down
// to 2^-28 of its largest weight, and a long flat tail below one dominating key is not lost.
template <int FMT> constexpr float kLift = FMT == kF32 ? 0.f : 15.f;
template <int FMT> constexpr float kFactor = FMT == kF32 ? 1.f : 1.f + 0x1p-11f;

struct HalfPair {
  uint32_t hi, lo;                                         // of two weights
};
__device__ __forceinline__ HalfPair split_weights(float a, float b) {
  constexpr float kShare = -(1.f - 0x1p-11f);
  const auto hi = __builtin_amdgcn_cvt_pkrtz(a, b);
  const auto lo = __builtin_amdgcn_cvt_pkrtz(fmaf((float)hi[0], kShare, a), fmaf((float)hi[1], kShare, b));
  return HalfPair{__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo)};
}

// All bits of the elements of a dword (one float, two halves, four 8-bit codes) that are infinite or NaN.
template <int FMT> __device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
  if constexpr (FMT == kF32) return (w & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
  constexpr uint32_t kMask = FMT == kF16 ? 0x7c007c00u : 0x7f7f7f7fu, kOne = FMT == kF16 ? 0x04000400u : 0x01010101u;
  const uint32_t top = ((w & kMask) + kOne) & (FMT == kF16 ? 0x80008000u : 0x80808080u);
  return top | (top - (top >> (FMT == kF16 ? 15 : 7)));
}

// Element e of the dwords that hold a lane's columns.
template <int FMT> __device__ __forceinline__ float element(const uint32_t* w, int e) {
  static_assert(FMT != kE2M1, "a block's scale says whether its elements are finite");
  if constexpr (FMT == kF32) return __uint_as_float(w[e]);
  const uint32_t pair = FMT == kF16 ? w[e >> 1] : (e & 2) ? codes_to_half2<true>(w[e >> 2]) : codes_to_half2<false>(w[e >> 2]);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(e & 1 ? pair >> 16 : pair));
}

// Four columns of the output: a row without weights gives zeros, whatever the values that it gave none.
template <int FMT, typename IO>
__device__ __forceinline__ void store_output(IO* out, float4_t o, float l) {
  const float norm = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) o = float4_t{0.f, 0.f, 0.f, 0.f};
  if constexpr (FMT == kF32)
    *reinterpret_cast<float4_t*>(out) = o * norm;
  else
    *reinterpret_cast<half4_t*>(out) =
        half4_t{(_Float16)(o[0] * norm), (_Float16)(o[1] * norm), (_Float16)(o[2] * norm), (_Float16)(o[3] * norm)};
}

// Four columns from d on of row rr of a segment, joined over the workgroup's waves:
// the output, or this workgroup's part.
template <int FMT, int D>
__device__ __forceinline__ void store_row(const AttnArgs& p, const SplitArgs& sp, const Segment& sg, bool complete, int rr,
                                          int d, float M, float l, float4_t o) {
  if (complete) {
    typedef typename std::conditional<FMT == kF32, float, _Float16>::type IO;
    const int row = sg.seg_row + rr, j = token_of(p, sg.s, row);
    IO* out = static_cast<IO*>(p.output) + ((int64_t)(sg.s.start + j) * p.Hq + sg.h * p.group + row - j * p.group) * D + d;
    store_output<FMT>(out, o, l);
  } else {
    float* part = sp.parts + (2 * (int64_t)sg.id + (sg.c0 == 0 ? 1 : 0)) * (sp.part_rows * (D + 2));
    *reinterpret_cast<float4_t*>(part + 2 * sp.part_rows + rr * D + d) = o;
    if (d == 0) {
      part[rr] = M;
      part[sp.part_rows + rr] = l;
    }
  }
}

template <int FMT, int D, int WAVES>
struct Shape {
  static constexpr int kBits = FMT == kF32 ? 32 : FMT == kF16 ? 16 : FMT == kE4M3 ? 8 : 4;   // of a cache element
  static constexpr int kRow = D * kBits / 8;                             // bytes of a position's k or v
  static constexpr int kBlocks = FMT == kF32 ? 1 : 2;                    // 16-position blocks of a wave's tile
  static constexpr int kTile = 16 * kBlocks;                             // positions of a tile
  static constexpr int kPos = 4 * kBlocks;                               // of them a lane group's
  static constexpr int kKWords = kRow < 64 ? kRow / 16 : 4;              // dwords of a load of k
  static constexpr int kKLoads = kRow / (16 * kKWords);                  // loads of a lane per block of k
  // columns of v a lane holds: sets of kCols neighbours, 16 * kCols apart
  static constexpr int kCols = FMT == kF32 ? 4 : FMT == kF16 ? (D / 16 < 8 ? D / 16 : 8) : D / 16;
  static constexpr int kSets = D / (16 * kCols);
  static constexpr int kSetBytes = kCols * kBits / 8;                    // of a set in one position
  static constexpr int kVWords = (kSetBytes + 3) / 4;                    // dwords of it
  static constexpr int kTileBytes = 2 * kTile * kRow;                    // of k and v
  // tiles a wave has in flight: 128 KiB a workgroup, at most 4. With 4 bits one: they are bound by what is done with
  // them, and more waves with fewer registers, in a loop of a quarter of the code, do that sooner (with 1, 2 and 4:
  // 64 requests of up to 16,384 positions, D = 128, 99, 101 and 114 us, D = 64 71, 78 and 88; 16 x 4 drafts of 6 heads
  // over 8,192, D = 256, 36, 38 and 43).
  static constexpr int kMostAhead = FMT == kE2M1 ? 1 : 4;
  static constexpr int kAhead = 131072 / WAVES / kTileBytes < kMostAhead ? 131072 / WAVES / kTileBytes : kMostAhead;
  static constexpr int kPitch = D + 4;                                   // floats between rows in LDS
};

constexpr int kStream = 2;                // cache policy of a buffer access: nontemporal

// BYTES: 4 for each word, or 2.
template <int POLICY, int BYTES, int WORDS>
__device__ __forceinline__ void load_words(rsrc_t rs, int offset, uint32_t (&w)[WORDS]) {
  if constexpr (BYTES == 2) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, offset, 0, POLICY);
  } else if constexpr (WORDS == 4) {
    const uint4_t x = __builtin_bit_cast(uint4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, offset, 0, POLICY));
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else if constexpr (WORDS == 2) {
    const uint2_t x = __builtin_bit_cast(uint2_t, __builtin_amdgcn_raw_buffer_load_b64(rs, offset, 0, POLICY));
    w[0] = x[0];
    w[1] = x[1];
  } else {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, offset, 0, POLICY);
  }
}

typedef const __attribute__((address_space(4))) int32_t* table_t;        // read through the scalar cache

// Where a request's positions of one key head lie. Positions come in aligned blocks of
// 16, which never cross a page.
template <bool LISTS>
struct Pages {
  const Args<LISTS>& p;
  table_t table, list;
  int h, end, newest;                                      // with lists: the list's positions, one past the token's own

  __device__ __forceinline__ explicit Pages(const Args<LISTS>& args)
      : p(args), table(nullptr), list(nullptr), h(0), end(0), newest(0) {}
  __device__ __forceinline__ void of(int r, int head, int past, int lane) {
    h = head;
    end = past;
    if constexpr (LISTS) {
      // the request that token r belongs to: those that end at or before it
      list = (table_t)(p.lists + ((int64_t)r * p.cache.Hk + head) * p.list_len);
      int owner = 0;
      if (p.owners.cu_seqlens == nullptr) {
        owner = min((int)((unsigned)r / (unsigned)p.owners.dense_len), p.owners.R - 1);
      } else {
        for (int first = 0; first < p.owners.R; first += 64) {
          const int i = first + lane;
          const int n = __builtin_popcountll(__ballot(i < p.owners.R && row_start(p.owners, min(i, p.owners.R - 1) + 1) <= r));
          owner += n;
          if (n < 64) break;
        }
        owner = __builtin_amdgcn_readfirstlane(min(owner, p.owners.R - 1));
      }
      const int64_t past_own = (int64_t)p.owners.seq_lens[owner] - row_start(p.owners, owner + 1) + r + 1;
      newest = (int)min(max(past_own, (int64_t)0), (int64_t)p.cache.max_pages << p.cache.page_shift);
      table = (table_t)(p.cache.table + (int64_t)owner * p.cache.max_pages);
    } else {
      table = (table_t)(p.cache.table + (int64_t)r * p.cache.max_pages);
    }
  }

  // The list's entry for the block at place pos of the list (any where pos is past it).
  __device__ __forceinline__ int listed(int pos) const {
    if constexpr (LISTS) return list[min(pos >> p.cache.page_shift, p.list_len - 1)];
    return 0;
  }
  // The position that the block at place pos begins at, or one past every table's end.
  __device__ __forceinline__ int first(int entry, int pos) const {
    return pos < end && (unsigned)entry < (unsigned)p.cache.max_pages
               ? (entry << p.cache.page_shift) + (pos & ((1 << p.cache.page_shift) - 1)) : 1 << 30;
  }

  // The table's entry for the block at pos (any entry where pos is past the table), to be checked below.
  __device__ __forceinline__ int entry(int pos) const {
    return table[min(pos >> p.cache.page_shift, p.cache.max_pages - 1)];
  }
  __device__ __forceinline__ int page(int entry, int pos) const {
    return (pos >> p.cache.page_shift) < p.cache.max_pages && entry < p.cache.num_pages ? entry : -1;
  }
  __device__ __forceinline__ int64_t row(int page, int pos) const {
    return (((int64_t)max(page, 0) * p.cache.Hk + h) << p.cache.page_shift) + (pos & ((1 << p.cache.page_shift) - 1));
  }
  // Rows of the block (or run of blocks) that exist: up to `end`, none without a page. Scalar, so that the resources made of it are.
  __device__ __forceinline__ int rows(int page, int pos, int most) const {
    return __builtin_amdgcn_readfirstlane(page >= 0 ? min(max((LISTS ? newest : end) - pos, 0), most) : 0);
  }
};

// Byte I of w at a float's exponent, in one instruction (the compiler takes a shift and a mask).
template <int I>
__device__ __forceinline__ uint32_t exponent_of(uint32_t w) {
  uint32_t x;
  const uint32_t by = 23;
  if constexpr (I == 0) asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0" : "=v"(x) : "v"(by), "v"(w));
  if constexpr (I == 1) asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1" : "=v"(x) : "v"(by), "v"(w));
  if constexpr (I == 2) asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2" : "=v"(x) : "v"(by), "v"(w));
  if constexpr (I == 3) asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3" : "=v"(x) : "v"(by), "v"(w));
  return x;
}

// WIDE: pages hold a whole tile (its two blocks share one look-up and one set of resources: with 4 bits, where the
// scalar unit's share of the time shows, and pages of 32 or more).
template <int FMT, int D, int WAVES, int TILES, bool LISTS, bool WIDE>
__global__ void __launch_bounds__(64 * WAVES, 1) gdn_attn_k(Args<LISTS> p, SplitArgs sp) {
  typedef Shape<FMT, D, WAVES> S;
  typedef typename std::conditional<FMT == kF32, float, _Float16>::type IO;
  constexpr int kAcc = S::kSets * S::kCols;                // 16 x 16 blocks of a row tile's output
  constexpr int kMost = TILES * kRows;                     // rows of a segment
  constexpr int U = S::kAhead;
  __shared__ alignas(16) float sums[WAVES][kMost][S::kPitch];
  __shared__ float stats[WAVES][kMost][2];
  __shared__ float joined[kMost][2];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  Share sh = find_share<LISTS>(p, sp, lane);
  // (with 4 bits it multiplies -inf, too, and must not be 0 there)
  float to_log2 = p.scale * 1.4426950408889634f;
  if (FMT == kE2M1 && to_log2 < 0x1p-126f) to_log2 = 0x1p-126f;
  const IO* __restrict__ qs = static_cast<const IO*>(p.q);
  if (tid == 0 && sp.notes != nullptr && sp.max_segs == 0) sp.notes[2 * sh.id] = int4{0, 0, 0, 0};
  bool again = false;
  // byte offsets of this lane in a block: 16 bytes of k in row n; its columns of v in rows 4 g + (0 .. 3)
  const int k_at = n * S::kRow + 4 * S::kKWords * g, v_at = 4 * g * S::kRow + S::kSetBytes * n;

  if (sh.u >= sh.u_end) return;
  int turn = blockIdx.x / kGroups;                         // see below
  Segment sg;
  Rows rw[TILES];                                          // of row 16 i + n
  Pages<LISTS> pages(p);
  int t = 0;
  half8_t qh[TILES][FMT == kF32 ? 1 : D / 32];             // q, the first product's second operand
  float4_t qf[TILES][FMT == kF32 ? D / 16 : 1];

  // ---- tiles: this wave's are t0 + (wave + WAVES i) kTile; U of them are in flight, tile i in buffer i % U.
  // A load past `end` or without a page has an empty range: it costs no traffic, and the number of
  // loads in flight stays the same, so that the wait for a tile waits for nothing younger.
  uint32_t kw[U][S::kBlocks][S::kKLoads][S::kKWords], vw[U][S::kPos][S::kSets][S::kVWords];
  // exponent bytes of this lane's positions; with e2m1, of the blocks of 32 elements that it holds
  constexpr int kScaleLoads = FMT == kE2M1 ? S::kKLoads : 1;
  uint32_t kscale[U][S::kBlocks][kScaleLoads], vscale[U][S::kBlocks];
  // table entries of the next tile, pages of this one; with lists the entries' numbers of the one after, and how many
  // positions a block of this one holds
  constexpr int kRun = WIDE ? S::kBlocks : 1, kFind = S::kBlocks / kRun;   // blocks that are looked up together, look-ups
  int entry[U][kFind], held[U][kFind];
  int pick[U][kFind], first_pos[U][kFind], block_pos[U][kFind], there_of[U][kFind];
  const int pos_mask = (1 << p.cache.page_shift) - 1;
  constexpr int kStep = WAVES * S::kTile;
  auto look_up = [&](int u, int t) {
#pragma unroll
    for (int a = 0; a < kFind; ++a) {
      if constexpr (LISTS) {
        first_pos[u][a] = pages.first(pick[u][a], t + 16 * kRun * a);
        entry[u][a] = pages.entry(first_pos[u][a]);
        pick[u][a] = pages.listed(t + U * kStep + 16 * kRun * a);
      } else {
        entry[u][a] = pages.entry(t + 16 * kRun * a);
      }
    }
  };
  // the scales of a page's head from row's slot on, all blocks of 32 (e2m1)
  auto scales_of = [&](const uint8_t* scales, int64_t row, int count) {
    return make_rsrc(scales + block_scale_at(row, 0, p.cache.page_shift, D),
                     count > 0 ? (D / 32 << p.cache.page_shift) - (int)(row & pos_mask) : 0);
  };
  auto load_k = [&](int u, int t) {
#pragma unroll
    for (int a = 0; a < kFind; ++a) {
      const int pos = LISTS ? first_pos[u][a] : t + 16 * kRun * a, page = pages.page(entry[u][a], pos);
      const int64_t row = pages.row(page, pos);
      const int count = pages.rows(page, pos, 16 * kRun);
      held[u][a] = page;
      if constexpr (LISTS) {
        block_pos[u][a] = pos;
        there_of[u][a] = count;
      }
      const rsrc_t rs = make_rsrc(static_cast<const char*>(p.cache.k) + row * S::kRow, count * S::kRow);
#pragma unroll
      for (int b = 0; b < kRun; ++b)
#pragma unroll
        for (int c = 0; c < S::kKLoads; ++c) load_words<0, 4>(rs, k_at + 64 * c + 16 * b * S::kRow, kw[u][kRun * a + b][c]);
      if constexpr (FMT == kE4M3)
        kscale[u][a][0] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.cache.k_scales + row, count > 0 ? 16 : 0), 4 * g, 0, 0);
      if constexpr (FMT == kE2M1) {
        // of row n, the block that holds this lane's elements
        const rsrc_t ss = scales_of(p.cache.k_scales, row, count);
#pragma unroll
        for (int b = 0; b < kRun; ++b)
#pragma unroll
          for (int c = 0; c < S::kKLoads; ++c)
            kscale[u][kRun * a + b][c] = __builtin_amdgcn_raw_buffer_load_b8(
                ss, ((4 * c + g * S::kKWords / 4) << p.cache.page_shift) + n + 16 * b, 0, 0);
      }
    }
  };
  auto load_v = [&](int u, int t) {
#pragma unroll
    for (int a = 0; a < kFind; ++a) {
      const int pos = LISTS ? block_pos[u][a] : t + 16 * kRun * a, page = held[u][a];
      const int64_t row = pages.row(page, pos);
      const int count = pages.rows(page, pos, 16 * kRun);
      const rsrc_t rs = make_rsrc(static_cast<const char*>(p.cache.v) + row * S::kRow, count * S::kRow);
#pragma unroll
      for (int b = 0; b < kRun; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < S::kSets; ++c)
            load_words<kStream, S::kSetBytes == 2 ? 2 : 4>(rs, v_at + (16 * b + e) * S::kRow + 16 * S::kSetBytes * c,
                                                           vw[u][4 * (kRun * a + b) + e][c]);
      if constexpr (FMT == kE2M1) {                        // of this lane's 4 positions, the block that holds its columns
        const rsrc_t ss = scales_of(p.cache.v_scales, row, count);
#pragma unroll
        for (int b = 0; b < kRun; ++b)
          vscale[u][kRun * a + b] = __builtin_amdgcn_raw_buffer_load_b32(
              ss, ((n * S::kCols / 32) << p.cache.page_shift) + 4 * g + 16 * b, 0, 0);
      }
      if constexpr (FMT == kE4M3)
        vscale[u][a] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.cache.v_scales + row, count > 0 ? 16 : 0), 4 * g, 0, 0);
    }
  };

  // The next segment: its q, then its first tiles, on their way while the last one's waves are joined.
  auto begin = [&]() {
    sg = next_segment<LISTS>(p, sp, sh);
    pages.of(sh.r, sg.h, sg.end, lane);
    t = sg.t0 + wave * S::kTile;
    if constexpr (LISTS) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int a = 0; a < kFind; ++a) pick[u][a] = pages.listed(t + u * kStep + 16 * kRun * a);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) look_up(u, t + u * kStep);
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      rw[i] = rows_of<LISTS>(p, sg.s, sg.seg_row, sg.rows, 16 * i + n);
      const IO* q = qs + (int64_t)(sg.s.start + rw[i].j) * p.q_stride + (int64_t)(sg.h * p.group + rw[i].head) * D;
      // in the order k is loaded in
      if constexpr (FMT == kF32) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) qf[i][c] = *reinterpret_cast<const float4_t*>(q + 16 * c + 4 * g);
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          qh[i][c] = *reinterpret_cast<const half8_t*>(
              q + (FMT == kF16 ? 32 * c + 8 * g
                   : FMT == kE4M3 || D == 64 ? 64 * (c >> 1) + 16 * g + 8 * (c & 1)
                                             : 128 * (c >> 2) + 32 * g + 8 * (c & 3)));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // in the order of the loop below: its waits count the younger loads on either way in
      __builtin_amdgcn_sched_barrier(0);
      load_k(u, t + u * kStep);
      __builtin_amdgcn_sched_barrier(0);
      load_v(u, t + u * kStep);
      look_up(u, t + (u + U) * kStep);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  begin();
  for (;;) {
    const int end = sg.end;
    int lo[TILES], hi[TILES];
    float4_t acc[TILES][kAcc];
    float M[TILES], l[TILES];                              // l: this lane's positions only
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      lo[i] = rw[i].lo;
      hi[i] = rw[i].hi;
      M[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kAcc; ++k) acc[i][k] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    bool some = t < end;
    while (some) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // Of the workgroups that share a CU, the oldest wave's instructions go first: their equal shares were done after
        // 66, 73 and 81 us (64 requests of up to 16,384 positions, D = 128; D = 64 33 to 50 us). Priorities that go
        // round, a tile each, make it 75 to 78 (40 to 48), the call 93.3 -> 90.4 us (66.3 -> 64.2).
        if (FMT == kE2M1 && TILES == 1 && sp.line_groups > kGroups) {
          if (turn & 2) {
            if (turn & 1) __builtin_amdgcn_s_setprio(3); else __builtin_amdgcn_s_setprio(2);
          } else {
            if (turn & 1) __builtin_amdgcn_s_setprio(1); else __builtin_amdgcn_s_setprio(0);
          }
          ++turn;
        }
        // ---- scores: block a of lane group g holds positions t + 16 a + 4 g + (0 .. 3)
        float4_t x[TILES][S::kBlocks];
#pragma unroll
        for (int a = 0; a < S::kBlocks; ++a) {
#pragma unroll
          for (int r = 0; r < TILES; ++r) x[r][a] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < S::kKLoads; ++c) {
            const uint32_t(&w)[S::kKWords] = kw[u][a][c];
            if constexpr (FMT == kF32) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int r = 0; r < TILES; ++r)
                  x[r][a] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]), qf[r][c][e], x[r][a], 0, 0, 0);
            } else if constexpr (FMT == kF16) {
#pragma unroll
              for (int r = 0; r < TILES; ++r)
                x[r][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                    __builtin_bit_cast(half8_t, uint4_t{w[0], w[1], w[2], w[3]}), qh[r][c], x[r][a], 0, 0, 0);
            } else if constexpr (FMT == kE2M1) {
              const float scale = __uint_as_float(kscale[u][a][c] << 23);
#pragma unroll
              for (int e = 0; e < S::kKWords; ++e) {
                const uint4_t v = uint4_t{nibbles_to_half2<0>(w[e], scale), nibbles_to_half2<1>(w[e], scale),
                                          nibbles_to_half2<2>(w[e], scale), nibbles_to_half2<3>(w[e], scale)};
#pragma unroll
                for (int r = 0; r < TILES; ++r)
                  x[r][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, v), qh[r][S::kKWords * c + e],
                                                                   x[r][a], 0, 0, 0);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint4_t v = uint4_t{codes_to_half2<false>(w[2 * e]), codes_to_half2<true>(w[2 * e]),
                                          codes_to_half2<false>(w[2 * e + 1]), codes_to_half2<true>(w[2 * e + 1])};
#pragma unroll
                for (int r = 0; r < TILES; ++r)
                  x[r][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, v), qh[r][2 * c + e], x[r][a],
                                                                   0, 0, 0);
              }
            }
          }
        }
        int page[kFind];                                   // of this tile: the next one's are looked up below
        int in_run[kFind];                                 // with lists, the positions of it that exist
        uint32_t ks[S::kBlocks];
#pragma unroll
        for (int a = 0; a < kFind; ++a) {
          page[a] = held[u][a];
          in_run[a] = LISTS ? there_of[u][a] : 16 * kRun;
        }
#pragma unroll
        for (int a = 0; a < S::kBlocks; ++a) ks[a] = FMT == kE4M3 ? kscale[u][a][0] : 0;
        // not before the products above: the loads then need registers of their own, and copies that wait
        // for them
        __builtin_amdgcn_sched_barrier(0);
        load_k(u, t + U * kStep);
        look_up(u, t + 2 * U * kStep);
        __builtin_amdgcn_sched_barrier(0);
        // to base-2 exponents. With 8-bit values the weight carries the value's scale, so xs is the
        // exponent of the product and `inv` takes the scale out of the weights' sum again; a zero row's
        // scale counts as 2^-33, below that of every other fp16 row.
        float xs[TILES][S::kPos], inv[S::kPos];
#pragma unroll
        for (int i = 0; i < S::kPos; ++i) {
          if constexpr (FMT == kE4M3) {
            const uint32_t kb = (ks[i >> 2] >> (8 * (i & 3))) & 255u;
            const uint32_t vb = max((vscale[u][i >> 2] >> (8 * (i & 3))) & 255u, 94u);
#pragma unroll
            for (int r = 0; r < TILES; ++r)
              xs[r][i] = fmaf(x[r][i >> 2][i & 3], to_log2 * __uint_as_float(kb << 23), (float)((int)vb - 127));
            inv[i] = __uint_as_float((254u - min(vb, 253u)) << 23);
          } else {
            // with 4 bits a score's distance from M takes the factor, below
#pragma unroll
            for (int r = 0; r < TILES; ++r) xs[r][i] = FMT == kE2M1 ? x[r][i >> 2][i & 3] : x[r][i >> 2][i & 3] * to_log2;
          }
        }

        // ---- masks, where some row does not attend all of the tile, or part of it has no page
        bool whole = t >= rw[0].lo_max && t + S::kTile <= rw[0].hi_min && t + S::kTile <= end;
#pragma unroll
        for (int a = 0; a < kFind; ++a) whole = whole && (LISTS ? in_run[a] == 16 * kRun : page[a] >= 0);
        bool mixed = false;                                // a non-finite value that only some rows attend
        if (__builtin_expect(!whole, 0)) {
#pragma unroll
          for (int i = 0; i < S::kPos; ++i) {
            const int pos = t + 16 * (i >> 2) + 4 * g + (i & 3);
            const int run = (i >> 2) / kRun;
            const bool there = LISTS ? 16 * ((i >> 2) % kRun) + 4 * g + (i & 3) < in_run[run] : page[run] >= 0 && pos < end;
#pragma unroll
            for (int r = 0; r < TILES; ++r)
              if (!(there && pos >= lo[r] && pos < hi[r])) xs[r][i] = -INFINITY;
            // a value that not every row attends may have to count for some: 0 times it has to be 0
            // for the others, whatever it is
            if (!(there && pos >= rw[0].lo_max && pos < rw[0].hi_min)) {
              if constexpr (FMT == kE2M1) {
                // a block is NaN by its scale; what lies beside a position that no row attends may be any byte
                const uint32_t sb = (vscale[u][i >> 2] >> (8 * (i & 3))) & 255u;
                if (sb > 140u) {
                  mixed = mixed || there;
                  vscale[u][i >> 2] &= ~(255u << (8 * (i & 3)));
#pragma unroll
                  for (int c = 0; c < S::kSets; ++c)
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) vw[u][i][c][w] = 0;
                }
                continue;
              }
#pragma unroll
              for (int c = 0; c < S::kSets; ++c)
#pragma unroll
                for (int w = 0; w < S::kVWords; ++w) {
                  const uint32_t bad = nonfinite<FMT>(vw[u][i][c][w]);
                  mixed = mixed || bad != 0;
                  vw[u][i][c][w] &= ~bad;
                }
            }
          }
          mixed = !LISTS && __any(mixed);                  // with lists all rows attend the same
        }

        // ---- weights
        float wgt[TILES][S::kPos];
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
          float m = xs[r][0];
          if constexpr (FMT == kE2M1) {
            // NaN where one is, which takes fewer instructions; M stays then, and l shows the NaN. M is a score as it is
            // here: its distance to another is exact where they are near, however large they are. (Score times factor less
            // a rounded M in one instruction is 0.3 % of a decode step and 1 % of drafts faster, but then M's rounding is
            // not the scores': weights of scores from 2^26 on left fp16's range.)
#pragma unroll
            for (int i = 1; i < S::kPos; ++i) m = __builtin_elementwise_maximum(m, xs[r][i]);
            m = __builtin_elementwise_maximum(row_maximum(m), M[r]);
          } else {
#pragma unroll
            for (int i = 1; i < S::kPos; ++i) m = fmaxf(m, xs[r][i]);
            m = fmaxf(row_max(m) - kLift<FMT>, M[r]);
          }
          if (__any(m > M[r])) {
            const float f = M[r] == m ? 1.f : exp2_fast(FMT == kE2M1 ? (M[r] - m) * to_log2 : M[r] - m);   // -inf - -inf is not asked for
            l[r] *= f;
#pragma unroll
            for (int i = 0; i < kAcc; ++i) acc[r][i] *= f;
            M[r] = m;
          }
          const float ref = M[r] == -INFINITY ? 0.f : M[r];
#pragma unroll
          for (int i = 0; i < S::kPos; ++i) {
            wgt[r][i] = exp2_fast(FMT == kE2M1 ? fmaf(xs[r][i] - ref, to_log2, kLift<FMT>) : xs[r][i] - ref);
            if constexpr (FMT == kE4M3)
              l[r] = fmaf(wgt[r][i], inv[i], l[r]);
            else
              l[r] += wgt[r][i];
          }
        }

        // ---- O^T += V^T P^T. A lane holds the same few columns of its 4 or 8 positions and turns them into
        // columns of positions with byte permutes (half an instruction an element).
        if constexpr (FMT == kF32) {
#pragma unroll
          for (int c = 0; c < S::kSets; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < TILES; ++r)
                  acc[r][4 * c + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vw[u][i][c][e]), wgt[r][i],
                                                                           acc[r][4 * c + e], 0, 0, 0);
        } else {
          // 32 positions a product
#pragma unroll
          for (int b = 0; b < S::kPos; b += 8) {
            float vs[8];                                   // e2m1: scales of this lane's columns
            if constexpr (FMT == kE2M1) {
#pragma unroll
              for (int a = 0; a < 2; ++a) {
                const uint32_t s = vscale[u][(b >> 2) + a];
                vs[4 * a] = __uint_as_float(exponent_of<0>(s));
                vs[4 * a + 1] = __uint_as_float(exponent_of<1>(s));
                vs[4 * a + 2] = __uint_as_float(exponent_of<2>(s));
                vs[4 * a + 3] = __uint_as_float(exponent_of<3>(s));
              }
            }
            uint4_t pw[TILES], pl[TILES];
#pragma unroll
            for (int r = 0; r < TILES; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const HalfPair w = split_weights(wgt[r][b + 2 * i], wgt[r][b + 2 * i + 1]);
                pw[r][i] = w.hi;
                pl[r][i] = w.lo;
              }
#pragma unroll
            for (int c = 0; c < S::kSets; ++c)
#pragma unroll
              for (int k = 0; k < S::kCols / 2; ++k) {     // two columns at a time
                uint32_t pair[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t(&w)[S::kVWords] = vw[u][b + i][c];
                  if constexpr (FMT == kF16)
                    pair[i] = w[k];
                  else if constexpr (FMT == kE2M1)
                    pair[i] = (k & 3) == 0   ? nibbles_to_half2<0>(w[k >> 2], vs[i])
                              : (k & 3) == 1 ? nibbles_to_half2<1>(w[k >> 2], vs[i])
                              : (k & 3) == 2 ? nibbles_to_half2<2>(w[k >> 2], vs[i])
                                             : nibbles_to_half2<3>(w[k >> 2], vs[i]);
                  else
                    pair[i] = (k & 1) ? codes_to_half2<true>(w[k >> 1]) : codes_to_half2<false>(w[k >> 1]);
                }
                uint4_t a0, a1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  a0[i] = __builtin_amdgcn_perm(pair[2 * i + 1], pair[2 * i], 0x05040100u);
                  a1[i] = __builtin_amdgcn_perm(pair[2 * i + 1], pair[2 * i], 0x07060302u);
                }
                const int o = S::kCols * c + 2 * k;
#pragma unroll
                for (int r = 0; r < TILES; ++r) {
                  const half8_t v0 = __builtin_bit_cast(half8_t, a0), v1 = __builtin_bit_cast(half8_t, a1);
                  const half8_t hi = __builtin_bit_cast(half8_t, pw[r]), lo = __builtin_bit_cast(half8_t, pl[r]);
                  acc[r][o] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, hi, acc[r][o], 0, 0, 0);
                  acc[r][o + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, hi, acc[r][o + 1], 0, 0, 0);
                  acc[r][o] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, lo, acc[r][o], 0, 0, 0);
                  acc[r][o + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, lo, acc[r][o + 1], 0, 0, 0);
                }
              }
          }
        }
        if (__builtin_expect(mixed, 0)) {
          // the values left out above, for the rows that attend them: position by position, element by
          // element, from memory
#pragma unroll 1
          for (int at = 0; at < S::kTile; ++at) {
            const int pos = t + at, pg = pages.page(pages.entry(pos & ~15), pos & ~15);
            if (pg < 0 || pos >= end) continue;
            float w[TILES];
            bool sees[TILES];
#pragma unroll
            for (int r = 0; r < TILES; ++r) {
              float own = wgt[r][0];
#pragma unroll
              for (int i = 1; i < S::kPos; ++i) own = 4 * (at >> 4) + (at & 3) == i ? wgt[r][i] : own;
              w[r] = __shfl(own, n + 16 * ((at >> 2) & 3));
              sees[r] = pos >= lo[r] && pos < hi[r] && !(pos >= rw[0].lo_max && pos < rw[0].hi_min);
            }
            if constexpr (FMT == kE2M1) {
              // a block's scale says it for all of the columns that a lane holds of it
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int block = S::kCols * (4 * g + i) / 32;
                if (p.cache.v_scales[block_scale_at(pages.row(pg, pos), block, p.cache.page_shift, D)] != 255) continue;
#pragma unroll
                for (int e = 0; e < S::kCols; ++e)
#pragma unroll
                  for (int r = 0; r < TILES; ++r)
                    if (sees[r]) acc[r][e][i] = NAN;
              }
            } else {
              const rsrc_t rs = make_rsrc(static_cast<const char*>(p.cache.v) + pages.row(pg, pos) * S::kRow, S::kRow);
#pragma unroll
              for (int c = 0; c < S::kSets; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  __builtin_amdgcn_sched_barrier(0);
                  uint32_t words[S::kVWords];
                  load_words<0, 4>(rs, S::kSetBytes * (16 * c + 4 * g + i), words);
#pragma unroll
                  for (int e = 0; e < S::kCols; ++e) {
                    const float v = element<FMT>(words, e);
#pragma unroll
                    for (int r = 0; r < TILES; ++r)
                      if (sees[r] && !(fabsf(v) < INFINITY))
                        acc[r][S::kCols * c + e][i] = fmaf(w[r], v, acc[r][S::kCols * c + e][i]);
                  }
                }
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_v(u, t + U * kStep);
        __builtin_amdgcn_sched_barrier(0);
        t += kStep;
        some = t < end;
        if (!some) break;                                  // short segments end here, past few of the steps
      }
    }

    const Segment done = sg;
    const int rows = done.rows;
    const bool complete = done.c0 == 0 && done.c1 == done.s.chunks;
    const bool more = sh.u < sh.u_end;
    if (more) begin();
    if (tid == 0 && sp.notes != nullptr && rows > 0 && done.c0 == 0 && (sp.max_segs > 0 || !complete)) note_segment(sp, done, sh);

    // ---- join the waves
    if (again) __syncthreads();                            // the last segment's sums have been read
    again = true;
#pragma unroll
    for (int r = 0; r < TILES; ++r) {
      if (FMT == kE2M1) M[r] *= to_log2;                   // from here on as the other formats', but for the lift
      l[r] = row_sum(l[r]) * kFactor<FMT>;
      if (l[r] != l[r]) M[r] = INFINITY;                   // a NaN score is no maximum, but has to show
      if (g == 0) {
        stats[wave][16 * r + n][0] = M[r];
        stats[wave][16 * r + n][1] = l[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < TILES; ++r) {
      const int rn = 16 * r + n;
      float top = stats[0][rn][0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = fmaxf(top, stats[w][rn][0]);
      const float f = M[r] == -INFINITY ? 0.f : exp2_fast(M[r] - top);
      if (tid < kRows) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
          total += stats[w][rn][0] == -INFINITY ? 0.f : stats[w][rn][1] * exp2_fast(stats[w][rn][0] - top);
        joined[rn][0] = top;
        joined[rn][1] = total;
      }
      // acc[cols c + e] of row n, register i: column 16 cols c + cols (4 g + i) + e
      if (rn < rows) {
#pragma unroll
        for (int c = 0; c < S::kSets; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < S::kCols; e += 4)
              *reinterpret_cast<float4_t*>(&sums[wave][rn][16 * S::kCols * c + S::kCols * (4 * g + i) + e]) =
                  float4_t{acc[r][S::kCols * c + e][i] * f, acc[r][S::kCols * c + e + 1][i] * f,
                           acc[r][S::kCols * c + e + 2][i] * f, acc[r][S::kCols * c + e + 3][i] * f};
      }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += 64 * WAVES) {
      const int rr = i / (D / 4), d = 4 * (i - rr * (D / 4));
      float4_t o = *reinterpret_cast<const float4_t*>(&sums[0][rr][d]);
#pragma unroll
      for (int w = 1; w < WAVES; ++w) o += *reinterpret_cast<const float4_t*>(&sums[w][rr][d]);
      store_row<FMT, D>(p, sp, done, complete, rr, d, joined[rr][0], joined[rr][1], o);
    }
    if (!more) return;
  }
}

// Joins the parts of the segments that several workgroups shared, as noted by the
// one that began them: a workgroup per note, kThreads / 16 / SLICES rows and 64
// columns, SLICES slices of 16 lanes taking alternate parts of a row. Parts are few
// and scattered, so latency counts: a slice loads several parts at once and joins
// them with a running M of its own.
template <int FMT, int D, int SLICES, bool LISTS>
__global__ void __launch_bounds__(kThreads) gdn_attn_join_k(Args<LISTS> p, SplitArgs sp) {
  typedef typename std::conditional<FMT == kF32, float, _Float16>::type IO;
  constexpr int kLanes = 16, kRowsHere = kThreads / kLanes / SLICES, kAhead = 4;
  __shared__ float4_t sums[kThreads];
  __shared__ float stats[kThreads / kLanes][2];
  const int tid = threadIdx.x, id = (int)blockIdx.x;
  const int4 a = sp.notes[2 * id], b = sp.notes[2 * id + 1];
  if constexpr (LISTS) {
    // notes by segment: those of tokens behind the last request are not written
    if (sp.max_segs > 0 && id / sp.max_segs / p.cache.Hk >= row_start(p.owners, p.owners.R)) return;
  }
  if (!LISTS && sp.max_segs > 0 && p.rows.cu_seqlens != nullptr) {
    // notes by segment: those of requests without that many rows are not written
    const int heads = sp.max_segs > 1 ? id / sp.max_segs : id, seg = id - heads * sp.max_segs, r = heads / p.cache.Hk;
    const int T = row_start(p.rows, r + 1) - row_start(p.rows, r);
    if ((int64_t)T * p.group <= (int64_t)seg << sp.seg_shift) return;
  }
  const int count = a.x, b0 = a.y, rows = a.z, seg_row = a.w, start = b.x, h = b.y;
  const int slot = tid / kLanes, slice = slot % SLICES;
  const int row0 = (int)blockIdx.y * kRowsHere, rr = row0 + slot / SLICES;
  if (count == 0 || row0 >= rows) return;
  const int64_t size = (int64_t)sp.part_rows * (D + 2);
  const int d = (int)blockIdx.z * 64 + 4 * (tid % kLanes), mine = min(rr, rows - 1);
  float4_t o = float4_t{0.f, 0.f, 0.f, 0.f};
  float M = -INFINITY, l = 0.f;
  for (int i = slice; i < count; i += SLICES * kAhead) {
    float m[kAhead], li[kAhead];
    float4_t x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // the first workgroup's part is its last segment, the others' their first; loads past
      // the last part repeat it
      const int at = min(i + k * SLICES, count - 1);
      const float* part = sp.parts + (2 * (int64_t)(b0 + at) + (at == 0 ? 1 : 0)) * size;
      m[k] = part[mine];
      li[k] = part[sp.part_rows + mine];
      x[k] = *reinterpret_cast<const float4_t*>(part + 2 * sp.part_rows + mine * D + d);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) top = i + k * SLICES < count ? fmaxf(top, m[k]) : top;
    const float f = M == -INFINITY ? 0.f : exp2_fast(M - top);
    o *= f;
    l *= f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool there = i + k * SLICES < count;
      const float w = there && m[k] != -INFINITY ? exp2_fast(m[k] - top) : 0.f;
      o += (there ? x[k] : float4_t{0.f, 0.f, 0.f, 0.f}) * w;   // 0 times a repeated part's infinity is NaN
      l = fmaf(li[k], w, l);
    }
    M = top;
  }
  sums[tid] = o;
  if (tid % kLanes == 0) {
    stats[slot][0] = M;
    stats[slot][1] = l;
  }
  __syncthreads();
  if (slice != 0 || rr >= rows) return;
  float top = M;
#pragma unroll
  for (int i = 1; i < SLICES; ++i) top = fmaxf(top, stats[slot + i][0]);
  o = float4_t{0.f, 0.f, 0.f, 0.f};
  l = 0.f;
#pragma unroll
  for (int i = 0; i < SLICES; ++i) {
    const float f = stats[slot + i][0] == -INFINITY ? 0.f : exp2_fast(stats[slot + i][0] - top);
    o += sums[tid + i * kLanes] * f;
    l = fmaf(stats[slot + i][1], f, l);
  }
  const int row = seg_row + rr, j = b.z == 1 ? 0 : (int)((unsigned)row / (unsigned)p.group);
  IO* out = static_cast<IO*>(p.output) + ((int64_t)(start + j) * p.Hq + h * p.group + row - j * p.group) * D + d;
  store_output<FMT>(out, o, l);
}

// Waves of gdn_attn_k's workgroups in a launch of at most one a CU: 8 with 16 KiB in
// flight each instead of 4 with 32, where a tile is 8 or 16 KiB and the registers suffice
// (a windowed FP32 step of 15 tokens 16.8 -> 15.5 us, 4 requests of 1,000 positions in 8
// bits 15.8 -> 14.4, one short request 9.3 -> 8.7; large ones within 1 %). With more
// workgroups than CUs two of 4 waves share one: 64 requests of 300 positions 17.6 us
// against 20.7, 256 of 1,000 172 against 198.
template <int FMT, int D, int TILES>
constexpr int many_waves() {
  typedef Shape<FMT, D, 8> S;
  const bool fits = TILES == 1 || (FMT != kE4M3 && FMT != kE2M1 && S::kRow <= 256);
  return fits && S::kAhead > 0 && 8 * S::kAhead * S::kTileBytes == 131072 && S::kTileBytes > 4096 ? 8 : 4;
}

// Workgroups of a split launch: one per CU keeps the waves' shares equal in time (of two
// on a CU the older one's loads go first: 64 requests of 8,192 positions, D = 128, the
// first 256 workgroups were done after 230 us and the others after 313), two where a
// wave's tiles in flight are small (8-bit heads of 64: 222 -> 195 us), and with 4 bits as
// many as the registers, or for two row tiles of 256 columns the LDS, let in.
template <int FMT, int D, int TILES>
constexpr int split_groups() {
  if (FMT == kE2M1) return (TILES == 1 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : D == 256 ? 1 : 2) * kGroups;
  typedef Shape<FMT, D, 4> S;
  return 4 * S::kAhead * S::kTileBytes < 131072 ? 2 * kGroups : kGroups;
}
constexpr int kMostGroups = 2 * kGroups, kMostGroups4 = 4 * kGroups;   // of a 4-bit cache

// Notes: two int4 each, one a workgroup or segment, at most the workgroups.
constexpr size_t kNoteBytes = (size_t)kMostGroups * 2 * sizeof(int4), kNoteBytes4 = (size_t)kMostGroups4 * 2 * sizeof(int4);

// Rows of a part: a segment's, of at most kTiles tiles.
int part_rows(int64_t N, int group) {
  const int64_t tiles = (N * group + kRows - 1) / kRows;
  return (int)(tiles < kTiles ? tiles : kTiles) * kRows;
}

// Whether every segment passes through one workgroup of its own, which spares the
// second launch (about 5 us with what it waits for). A workgroup alone takes in about
// 47 KB a us (of 8-bit pages 29, which it has to turn into halves); split evenly, the
// whole call runs at about 6.4 GB a ms. Half of that time is what the longest segment
// may take before the others wait for it. Measured, whole against split: 64 requests of
// 1,000 positions, 8 key heads of 128 fp16 47 and 49 us, 16 of 600 13 and 18, one of 333
// 8.3 and 9.4, of 700 12.7 and 9.3, 4 of 1,000 in 8 bits 14.3 and 10.8; 16 of 2,048 with
// 4 heads 28 and 18 us. 4-bit pages are taken in at 110 to 160 positions a us, of any
// width: one of 1,000, 8 heads of 128, 12.1 and 8.5 us, 64 of 2,000 29.6 and 34.4; 64 of
// 1,000, 4 heads of 256, 17.4 and 21.1. Without the host's lengths the sum is not known and counts as
// nothing.
template <int FMT, int D>
bool one_group_each(int64_t longest, int64_t sum, int heads, int64_t position_bytes) {
  constexpr double kRate = FMT == kE2M1 ? (D == 256 ? 29e3 : D == 128 ? 20e3 : 10e3) : FMT == kE4M3 ? 29e3 : 47e3;
  const double alone = (double)longest * position_bytes / kRate;
  const double together = (double)sum * heads * position_bytes / 6.4e6;
  return alone <= together / 2 + 5.0;
}

// Units of kChunkShift positions that a segment's beginning and joining count as where 4-bit lengths are split, so that
// workgroups with two segments are not the last: one, or with two row tiles two. Not where few workgroups hold two
// or shares are one or two units, which a unit more rounds up for all. Without and with, on the same buffers: 16 x up to 4
// drafts of 6 heads over up to 8,191 positions, D = 256, 34.1 and 31.5 us, 64 x 4 over 8,192 81.3 and 78.3; 64 requests of
// up to 2,000, 8 heads of 128, 22.8 and 21.1 (4 of 256 22.2 and 22.6), of up to 16,384 94.0 and 93.3. Where the rule leaves
// it out, 1 x 4 over 8,191, it was 15.9 and 17.3.
// Nor where all segments' units would not fit kMostUnits, however many positions one holds.
inline int fixed_part(int tiles, int64_t segments, int64_t positions, int64_t rows, int64_t groups) {
  const double units = (double)positions * (double)((rows + tiles * kRows - 1) / (tiles * kRows)) / (1 << kChunkShift);
  return segments * 8 >= groups && units >= 2.0 * (double)groups && segments * (1 + tiles) <= kMostUnits ? tiles : 0;
}

template <int FMT, int D, int TILES, bool LISTS, bool WIDE>
void launch_few(const Args<LISTS>& p, const SplitArgs& sp, int groups, hipStream_t stream) {
  if constexpr (FMT == kE2M1 && !WIDE) {
    if (p.cache.page_shift >= 5) return launch_few<FMT, D, TILES, LISTS, true>(p, sp, groups, stream);
  }
  constexpr int kMany = many_waves<FMT, D, TILES>();
  if (groups <= kGroups)
    hipLaunchKernelGGL((gdn_attn_k<FMT, D, kMany, TILES, LISTS, WIDE>), dim3((unsigned)groups), dim3(64 * kMany), 0, stream, p, sp);
  else
    hipLaunchKernelGGL((gdn_attn_k<FMT, D, 4, TILES, LISTS, WIDE>), dim3((unsigned)groups), dim3(256), 0, stream, p, sp);
}

template <int FMT, int D, bool LISTS>
hipError_t launch_attn_d(const Args<LISTS>& p, void* workspace, hipStream_t stream) {
  SplitArgs sp{};
  const int64_t most = (int64_t)p.max_tokens * p.group;    // rows of a request and key head
  const bool few = most <= kRows;
  const int seg_rows = few ? kRows : kTiles * kRows;
  sp.seg_shift = few ? 4 : 5;
  static_assert(kRows == 16 && kTiles == 2, "see seg_shift");
  const int64_t segments = ((most <= seg_rows ? 0 : (int64_t)p.rows.N * p.group / seg_rows) + p.rows.R) * p.cache.Hk;
  int64_t groups = segments;
  const bool whole = one_group_each<FMT, D>(p.max_len, p.sum_len, p.cache.Hk, 2 * Shape<FMT, D, 4>::kRow);
  int64_t notes = 0;
  int64_t cap = (int64_t)p.cache.max_pages << p.cache.page_shift;
  if constexpr (LISTS) cap = (int64_t)p.list_len << p.cache.page_shift;
  if (whole && (segments <= kOneEach || segments > kMostShared)) {
    sp.chunk_shift = kWholeShift;
    if (segments > kMostShared) groups = 2 * kGroups;      // evenly by their number: units are counted in 32 bits
  } else if (whole) {
    groups = 2 * kGroups;
    sp.chunk_shift = 5;
    sp.whole = 1;
    sp.more = (FMT == kE2M1 ? kSegmentBytes4 : kSegmentBytes) / (32 * 2 * Shape<FMT, D, 4>::kRow);
    while (segments * ((cap >> sp.chunk_shift) + 1 + sp.more) > kMostUnits) ++sp.chunk_shift;
  } else {
    static_assert(FMT == kE2M1 || split_groups<FMT, D, 1>() == (D == 64 ? split_groups<FMT, 64, 1>() : kGroups),
                  "see attn_workspace_bytes");
    groups = few ? split_groups<FMT, D, 1>() : split_groups<FMT, D, kTiles>();
    sp.notes = static_cast<int4*>(workspace);
    sp.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + (FMT == kE2M1 ? kNoteBytes4 : kNoteBytes));
    sp.part_rows = few ? kRows : part_rows(p.rows.N, p.group);
    sp.chunk_shift = kChunkShift;
    if constexpr (FMT == kE2M1) sp.more = fixed_part(few ? 1 : kTiles, segments, p.sum_len * p.cache.Hk, most, groups);
    while (segments * ((cap >> sp.chunk_shift) + 1 + sp.more) > kMostUnits) ++sp.chunk_shift;
    // notes by segment where there are fewer segments than workgroups
    const int64_t segs = (most + seg_rows - 1) / seg_rows;
    notes = segs * p.rows.R * p.cache.Hk;
    if (notes <= groups) sp.max_segs = (int)segs; else notes = groups;
    if (segs > 1 && segs <= kMostLines && ((int64_t)p.rows.N * p.group / p.rows.R + seg_rows - 1) / seg_rows == segs)
      while (1 << sp.line_shift < segs) ++sp.line_shift;
  }
  sp.line_groups = (int)groups >> sp.line_shift;
  if (few)
    launch_few<FMT, D, 1, LISTS, false>(p, sp, (int)groups, stream);
  else
    launch_few<FMT, D, kTiles, LISTS, false>(p, sp, (int)groups, stream);
  if (!whole) {
    // 16 slices where a segment has more than 16 parts on average, else 2
    const unsigned rows = (unsigned)(most < seg_rows ? most : seg_rows);
    if (notes * 16 < groups)
      hipLaunchKernelGGL((gdn_attn_join_k<FMT, D, 16, LISTS>), dim3((unsigned)notes, rows, D / 64), dim3(kThreads), 0, stream, p, sp);
    else
      hipLaunchKernelGGL((gdn_attn_join_k<FMT, D, 2, LISTS>), dim3((unsigned)notes, (rows + 7) / 8, D / 64), dim3(kThreads), 0,
                         stream, p, sp);
  }
  return hipGetLastError();
}

template <int FMT, bool LISTS>
hipError_t launch_attn_f(const Args<LISTS>& p, void* workspace, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_attn_d<FMT, 64, LISTS>(p, workspace, stream);
    case 128: return launch_attn_d<FMT, 128, LISTS>(p, workspace, stream);
    case 256: return launch_attn_d<FMT, 256, LISTS>(p, workspace, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace gdn

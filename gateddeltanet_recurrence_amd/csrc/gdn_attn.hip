// Attention of every request's newest tokens over its paged cache:
// gdn_attn_forward.
//
// With the scores x_t = scale log2(e) q.k_t of the attended positions, a row's
// output is sum_t 2^(x_t - M) v_t / sum_t 2^(x_t - M) for any M. A wave walks its
// positions once with a running M (the largest x so far), l (the sum of the
// weights) and the output's unnormalised sum, rescaling both when M grows; waves,
// and workgroups that share a request's length, are joined by the same rule.
//
// Decode reads every key and value once for at most 16 rows (tokens x heads of a
// key head), so it is bound by HBM; the matrix cores only keep the arithmetic out
// of the way. The layouts follow from loading both operands straight into
// registers, with no LDS and no barrier in the loop:
//  - rows are the N side of both products: S^T = K Q^T and O^T = V^T P^T. A row's
//    scores then lie in 4 lanes (l & 15 = row), its weights leave the first
//    product in the order the second one takes them in, and the running M, l and
//    the rescaling factor are one register each.
//  - a wave's tile is 32 positions (16 for fp32). Lane group g = l >> 4 takes the
//    positions 8 g .. 8 g + 7 in the second product's contraction, so the first
//    product's two 16-position blocks hold the positions 8 g + 4 a + (0 .. 3).
//  - v is loaded in rows too: a lane holds the same few columns of 8 positions and
//    turns them into columns with byte permutes (half an instruction an element).
//
// Rows come in tiles of 16, and a workgroup takes up to 4 tiles of a request and key
// head: with one tile its 4 waves take alternate positions, with two tiles 2 waves
// each, with more one wave each. Waves of different tiles then read the same keys and
// values at the same time, through one CU's L1, so HBM is read once for up to 64 rows.
//
// Work is split evenly over the workgroups whatever the lengths: the positions of
// every (request, group of tiles, key head) in chunks of 128 are laid end to end, and
// workgroup b takes the b-th equal share of the chunks. A share that holds all of a
// segment's chunks writes the output; the others leave (M, l, sum) in the workspace
// and gdn_attn_join_k, a second launch, joins them. Every workgroup forms the
// prefix sums of the requests' chunks by itself: R loads and one scan instead of a
// launch. The order of every sum is fixed by the lengths, so results repeat bit for
// bit; no atomics are used.
#include <type_traits>

#include "gdn_attn_kernels.h"
#include "gdn_common.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 16;                 // rows of a tile: the N side of the MFMA
constexpr int kTiles = 4;                 // tiles of a workgroup
constexpr int kChunkShift = 7;            // positions of a unit of work: 128
constexpr int kWholeShift = 30;           // one unit per segment: nothing is split
constexpr int kGroups = 512;              // workgroups of a split launch: two per CU

enum Format { kF32 = 0, kF16 = 1, kE4M3 = 2 };

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

struct SplitArgs {
  int64_t* prefix;                        // [R + 1] chunks before a request; null: nothing is split
  float* parts;                           // [2 * groups][part_rows * (D + 2)]: M, l, sums
  int32_t part_rows;
  int32_t chunk_shift;
};

// What a request brings: its rows, the positions any of them attends and its units.
struct Plan {
  int start, T;                           // first token, tokens
  int64_t len;                            // seq_lens[r] as given
  int base, hi;                           // positions [base, hi), base a multiple of 32
  int segs, chunks;                       // groups of kTiles tiles, units of each
};

__device__ __forceinline__ int clamp_pos(int64_t x, int hi) { return (int)(x < 0 ? 0 : x > hi ? hi : x); }

__device__ __forceinline__ Plan plan_of(const AttnArgs& p, int r, int chunk_shift) {
  Plan s;
  s.start = row_start(p.rows, r);
  s.T = max(row_start(p.rows, r + 1) - s.start, 0);
  s.len = p.rows.seq_lens[r];
  const int cap = p.cache.max_pages << p.cache.page_shift;
  s.hi = clamp_pos(s.len, cap);
  s.base = p.window > 0 ? clamp_pos(s.len - s.T + 1 - p.window, s.hi) & ~31 : 0;
  s.segs = (s.T * p.group + kTiles * kRows - 1) / (kTiles * kRows);
  s.chunks = s.T > 0 ? max((int)(((int64_t)s.hi - s.base + (1ll << chunk_shift) - 1) >> chunk_shift), 1) : 0;
  return s;
}

__device__ __forceinline__ int64_t units_of(const Plan& s, int Hk) { return (int64_t)s.segs * Hk * s.chunks; }

__device__ __forceinline__ int64_t share_of(int64_t total, int groups) { return max((total + groups - 1) / groups, (int64_t)1); }

// Largest (sum) over the 4 lanes that hold a row: l & 15 the same.
__device__ __forceinline__ float row_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
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

template <int FMT> __device__ __forceinline__ bool any_nonfinite(uint32_t w) {
  if constexpr (FMT == kF16) return (((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u) != 0;
  if constexpr (FMT == kE4M3) return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
  return (w & 0x7f800000u) == 0x7f800000u;
}

template <int FMT, int D>
struct Shape {
  static constexpr int kBytes = FMT == kF32 ? 4 : FMT == kF16 ? 2 : 1;   // of a cache element
  static constexpr int kTile = FMT == kF32 ? 16 : 32;                    // positions of a wave's tile
  static constexpr int kBlocks = kTile / 16;                             // 16-position blocks of the first product
  static constexpr int kPos = kTile / 4;                                 // positions of a lane group: 4 or 8
  static constexpr int kKLoads = D * kBytes / 64;                        // 16-byte loads of a lane per block of k
  // columns of v a lane holds: sets of kCols neighbours, 16 * kCols apart
  static constexpr int kCols = FMT == kF32 ? 4 : FMT == kF16 ? (D / 16 < 8 ? D / 16 : 8) : D / 16;
  static constexpr int kSets = D / (16 * kCols);
  static constexpr int kVWords = kCols * kBytes / 4;                     // dwords of a set in one position
  static constexpr int kPitch = D + 4;                                   // floats between rows in LDS
};

template <int WORDS>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 4) {
    const uint4_t x = __builtin_nontemporal_load(reinterpret_cast<const uint4_t*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else if constexpr (WORDS == 2) {
    const uint2_t x = __builtin_nontemporal_load(reinterpret_cast<const uint2_t*>(p));
    w[0] = x[0];
    w[1] = x[1];
  } else {
    w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  }
}

// The page-table entry of a position, or -1. The position is below 2^30.
__device__ __forceinline__ int page_of(const AttnArgs& p, const int32_t* table, int pos) {
  const int i = pos >> p.cache.page_shift;
  const int page = i < p.cache.max_pages ? table[i] : -1;
  return page < p.cache.num_pages ? page : -1;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, D == 256 && FMT == kF32 ? 1 : 2) gdn_attn_k(AttnArgs p, SplitArgs sp) {
  typedef Shape<FMT, D> S;
  typedef typename std::conditional<FMT == kF32, float, _Float16>::type IO;
  constexpr int kAcc = S::kSets * S::kCols;                // 16 x 16 blocks of the output
  __shared__ alignas(16) float sums[kWaves][kRows][S::kPitch];
  __shared__ float stats[kWaves][kRows][2];
  __shared__ int64_t scan[kWaves + 1];
  __shared__ int64_t first[2];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;

  // ---- this workgroup's share of the units
  const int per = (p.rows.R + kThreads - 1) / kThreads;    // requests a thread sums
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < p.rows.R) mine += units_of(plan_of(p, r, sp.chunk_shift), p.cache.Hk);
  }
  int64_t before = mine;                                   // inclusive scan over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t x = __shfl_up(before, d);
    if (lane >= d) before += x;
  }
  if (lane == 63) scan[wave] = before;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  before -= mine;
  const int64_t share = share_of(total, (int)gridDim.x);
  int64_t u = (int64_t)blockIdx.x * share;
  const int64_t u_end = min(u + share, total);
  {
    int64_t at = before;
    if (mine > 0 && u >= before && u < before + mine) {
      for (int i = 0; i < per; ++i) {
        const int64_t x = units_of(plan_of(p, tid * per + i, sp.chunk_shift), p.cache.Hk);
        if (u < at + x) {
          first[0] = tid * per + i;
          first[1] = at;
          break;
        }
        at += x;
      }
    }
    if (blockIdx.x == 0 && sp.prefix != nullptr) {
      at = before;
      for (int i = 0; i < per; ++i) {
        const int r = tid * per + i;
        if (r < p.rows.R) {
          sp.prefix[r] = at;
          at += units_of(plan_of(p, r, sp.chunk_shift), p.cache.Hk);
        }
      }
      if (tid == 0) sp.prefix[p.rows.R] = total;
    }
  }
  __syncthreads();
  if (u >= u_end) return;
  int r = __builtin_amdgcn_readfirstlane((int)first[0]);
  int64_t r_first = first[1];

  const float to_log2 = p.scale * 1.4426950408889634f;
  const IO* __restrict__ qs = static_cast<const IO*>(p.q);

  while (u < u_end) {
    // ---- the next segment: chunks [c0, c1) of (request, tile, key head)
    Plan s = plan_of(p, r, sp.chunk_shift);
    while (u - r_first >= units_of(s, p.cache.Hk)) {       // requests without tokens have no units
      r_first += units_of(s, p.cache.Hk);
      s = plan_of(p, ++r, sp.chunk_shift);
    }
    const int64_t local = u - r_first;
    const int seg = __builtin_amdgcn_readfirstlane((int)(local / s.chunks));
    const int c0 = __builtin_amdgcn_readfirstlane((int)(local - (int64_t)seg * s.chunks));
    const int c1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)s.chunks, c0 + (u_end - u)));
    const int h = seg / s.segs, seg_row = (seg - h * s.segs) * (kTiles * kRows);
    u += c1 - c0;

    // ---- the wave's tile and stream of positions, this lane's row, and what the tile's rows attend
    const int seg_rows = min(kTiles * kRows, s.T * p.group - seg_row);
    const int streams = seg_rows <= kRows ? 4 : seg_rows <= 2 * kRows ? 2 : 1;
    const int sub = wave / streams, stream = wave - sub * streams;
    const int rows = max(min(kRows, seg_rows - sub * kRows), 0);       // 0: a wave without a tile
    const int row0 = seg_row + (rows > 0 ? sub * kRows : 0), last_row = row0 + max(rows, 1) - 1;
    const int cap = p.cache.max_pages << p.cache.page_shift;
    const int row = min(row0 + n, last_row);
    const int j = row / p.group;
    const int64_t past = s.len - s.T + j + 1;              // one past the row's newest position
    const int hi = n < rows ? clamp_pos(past, cap) : 0;
    const int lo = p.window > 0 ? clamp_pos(past - p.window, cap) : 0;
    const int64_t past0 = s.len - s.T + row0 / p.group + 1, past1 = s.len - s.T + last_row / p.group + 1;
    const int hi_min = clamp_pos(past0, cap), hi_max = rows > 0 ? clamp_pos(past1, cap) : 0;
    const int lo_min = p.window > 0 ? clamp_pos(past0 - p.window, cap) : 0;
    const int lo_max = p.window > 0 ? clamp_pos(past1 - p.window, cap) : 0;
    const int t0 = s.base + (int)((int64_t)c0 << sp.chunk_shift);
    const int t1 = (int)min((int64_t)s.base + ((int64_t)c1 << sp.chunk_shift), (int64_t)hi_max);
    const int step = streams * S::kTile;

    // q as the first product's second operand, in the order k is loaded in
    const IO* q = qs + (int64_t)(s.start + j) * p.q_stride + (int64_t)(h * p.group + row - j * p.group) * D;
    half8_t qh[FMT == kF32 ? 1 : D / 32];
    float4_t qf[FMT == kF32 ? D / 16 : 1];
    if constexpr (FMT == kF32) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) qf[c] = *reinterpret_cast<const float4_t*>(q + 16 * c + 4 * g);
    } else {
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        qh[c] = *reinterpret_cast<const half8_t*>(
            q + (FMT == kF16 ? 32 * c + 8 * g : 64 * (c >> 1) + 16 * g + 8 * (c & 1)));
    }

    float4_t acc[kAcc];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    float M = -INFINITY, l = 0.f;                          // l: this lane's positions only

    const int32_t* table = p.cache.table + (int64_t)r * p.cache.max_pages;
    const int in_page = (1 << p.cache.page_shift) - 1;
    // positions this lane loads: k of block a at kpos + 4 a (fp32: kpos), v at vpos + 0 .. kPos - 1
    const int kpos = FMT == kF32 ? n : 8 * (n >> 2) + (n & 3), vpos = S::kPos * g;

    int kpage = -1, vpage = -1;
    int t = t0 + stream * S::kTile;
    if (t < t1) {
      kpage = page_of(p, table, t + kpos);
      vpage = page_of(p, table, t + vpos);
    }
    for (; t < t1; t += step) {
      const bool held = vpage >= 0;
      const int64_t krow = (((int64_t)max(kpage, 0) * p.cache.Hk + h) << p.cache.page_shift) + ((t + kpos) & in_page);
      const int64_t vrow = (((int64_t)max(vpage, 0) * p.cache.Hk + h) << p.cache.page_shift) + ((t + vpos) & in_page);
      const char* kp = static_cast<const char*>(p.cache.k) + krow * (D * S::kBytes) + 16 * g;
      const char* vp = static_cast<const char*>(p.cache.v) + vrow * (D * S::kBytes) + S::kCols * S::kBytes * n;
      uint32_t kw[S::kBlocks][S::kKLoads][4];
#pragma unroll
      for (int a = 0; a < S::kBlocks; ++a)
#pragma unroll
        for (int c = 0; c < S::kKLoads; ++c) load_words(kp + 4 * a * D * S::kBytes + 64 * c, kw[a][c]);
      uint2 kscale, vscale;                                // exponent bytes of this lane group's 8 positions
      if constexpr (FMT == kE4M3) {
        kscale = *reinterpret_cast<const uint2*>(p.cache.k_scales + vrow);
        vscale = *reinterpret_cast<const uint2*>(p.cache.v_scales + vrow);
      }
      uint32_t vw[S::kPos][S::kSets][S::kVWords];
#pragma unroll
      for (int i = 0; i < S::kPos; ++i)
#pragma unroll
        for (int c = 0; c < S::kSets; ++c)
          load_words(vp + (i * D + 16 * S::kCols * c) * S::kBytes, vw[i][c]);
      const int next = t + step;
      if (next < t1) {
        kpage = page_of(p, table, next + kpos);
        vpage = page_of(p, table, next + vpos);
      }

      // ---- scores: block a of lane group g holds positions t + kPos g + 4 a + (0 .. 3)
      float4_t x[S::kBlocks];
#pragma unroll
      for (int a = 0; a < S::kBlocks; ++a) {
        x[a] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < S::kKLoads; ++c) {
          if constexpr (FMT == kF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[a] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kw[a][c][e]), qf[c][e], x[a], 0, 0, 0);
          } else if constexpr (FMT == kF16) {
            const uint4_t w = uint4_t{kw[a][c][0], kw[a][c][1], kw[a][c][2], kw[a][c][3]};
            x[a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w), qh[c], x[a], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4_t w = uint4_t{codes_to_half2<false>(kw[a][c][2 * e]), codes_to_half2<true>(kw[a][c][2 * e]),
                                        codes_to_half2<false>(kw[a][c][2 * e + 1]),
                                        codes_to_half2<true>(kw[a][c][2 * e + 1])};
              x[a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w), qh[2 * c + e], x[a], 0, 0, 0);
            }
          }
        }
      }
      // to base-2 exponents. With 8-bit values the weight carries the value's scale, so x is the
      // exponent of the product and `inv` takes the scale out of the weights' sum again; a zero row's
      // scale counts as 2^-33, below that of every other fp16 row.
      float xs[S::kPos], inv[S::kPos];
#pragma unroll
      for (int i = 0; i < S::kPos; ++i) {
        if constexpr (FMT == kE4M3) {
          const uint32_t kb = ((i < 4 ? kscale.x : kscale.y) >> (8 * (i & 3))) & 255u;
          const uint32_t vb = max(((i < 4 ? vscale.x : vscale.y) >> (8 * (i & 3))) & 255u, 94u);
          xs[i] = fmaf(x[i >> 2][i & 3], to_log2 * __uint_as_float(kb << 23), (float)((int)vb - 127));
          inv[i] = __uint_as_float((254u - min(vb, 253u)) << 23);
        } else {
          xs[i] = x[i >> 2][i & 3] * to_log2;
        }
      }

      // ---- masks, where the tile reaches past what every row attends or has no page
      const bool whole = t >= lo_max && t + S::kTile <= hi_min && __all(held);
      bool mixed = false;                                  // a non-finite value that only some rows attend
      if (!whole) {
#pragma unroll
        for (int i = 0; i < S::kPos; ++i) {
          const int pos = t + vpos + i;
          if (!(held && pos >= lo && pos < hi)) xs[i] = -INFINITY;
          const bool any = held && pos >= lo_min && pos < hi_max, all = held && pos >= lo_max && pos < hi_min;
#pragma unroll
          for (int c = 0; c < S::kSets; ++c)
#pragma unroll
            for (int w = 0; w < S::kVWords; ++w) {
              if (!any) vw[i][c][w] = 0;                   // whatever lies there, 0 times it has to be 0
              if (any && !all) mixed = mixed || any_nonfinite<FMT>(vw[i][c][w]);
            }
        }
        mixed = __any(mixed);
      }

      // ---- weights
      float m = xs[0];
#pragma unroll
      for (int i = 1; i < S::kPos; ++i) m = fmaxf(m, xs[i]);
      m = fmaxf(row_max(m), M);
      if (__any(m > M)) {
        const float f = M == m ? 1.f : exp2_fast(M - m);   // -inf - -inf is not asked for
        l *= f;
#pragma unroll
        for (int i = 0; i < kAcc; ++i) acc[i] *= f;
        M = m;
      }
      const float ref = M == -INFINITY ? 0.f : M;
      float wgt[S::kPos];
#pragma unroll
      for (int i = 0; i < S::kPos; ++i) {
        wgt[i] = exp2_fast(xs[i] - ref);
        if constexpr (FMT == kE4M3)
          l = fmaf(wgt[i], inv[i], l);
        else
          l += wgt[i];
      }

      // ---- O^T += V^T P^T
      half8_t pw;
      if constexpr (FMT != kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pw[i] = (_Float16)wgt[i];
      }
      // `seen`: a mask per position of what to keep of v; the sums of lanes with keep false stay
      auto product = [&](auto all, const uint32_t (&seen)[S::kPos], bool keep) {
        constexpr bool kAll = decltype(all)::value;
        auto add = [&](int o, const float4_t& x) {
          if constexpr (kAll) {
            acc[o] = x;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[o][e] = keep ? x[e] : acc[o][e];
          }
        };
        if constexpr (FMT == kF32) {
#pragma unroll
          for (int c = 0; c < S::kSets; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float4_t x = acc[4 * c + e];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    __uint_as_float(kAll ? vw[i][c][e] : vw[i][c][e] & seen[i]), wgt[i], x, 0, 0, 0);
              add(4 * c + e, x);
            }
        } else {
#pragma unroll
          for (int c = 0; c < S::kSets; ++c)
#pragma unroll
            for (int q2 = 0; q2 < S::kCols / 2; ++q2) {    // two columns at a time
              uint32_t pair[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if constexpr (FMT == kF16)
                  pair[i] = vw[i][c][q2];
                else
                  pair[i] = (q2 & 1) ? codes_to_half2<true>(vw[i][c][q2 >> 1]) : codes_to_half2<false>(vw[i][c][q2 >> 1]);
                if constexpr (!kAll) pair[i] &= seen[i];
              }
              uint4_t a0, a1;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a0[i] = __builtin_amdgcn_perm(pair[2 * i + 1], pair[2 * i], 0x05040100u);
                a1[i] = __builtin_amdgcn_perm(pair[2 * i + 1], pair[2 * i], 0x07060302u);
              }
              const int o = S::kCols * c + 2 * q2;
              add(o, __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a0), pw, acc[o], 0, 0, 0));
              add(o + 1, __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a1), pw, acc[o + 1], 0, 0, 0));
            }
        }
      };
      uint32_t seen[S::kPos] = {};
      if (!mixed) {
        product(std::true_type{}, seen, true);
      } else {
        // a row at a time, with the values it does not attend taken out
#pragma unroll 1
        for (int k = 0; k < rows; ++k) {
          const int row_hi = __shfl(hi, k), row_lo = __shfl(lo, k);
#pragma unroll
          for (int i = 0; i < S::kPos; ++i) {
            const int pos = t + vpos + i;
            seen[i] = pos >= row_lo && pos < row_hi ? 0xffffffffu : 0u;
          }
          product(std::false_type{}, seen, n == k);
        }
      }
    }

    // ---- join the waves
    l = row_sum(l);
    __syncthreads();                                       // the last segment's sums have been read
    if (g == 0) {
      stats[wave][n][0] = M;
      stats[wave][n][1] = l;
    }
    __syncthreads();
    const int w0 = sub * streams;                          // the waves of this wave's tile
    float top = M;
    for (int w = w0; w < w0 + streams; ++w) top = fmaxf(top, stats[w][n][0]);
    const float f = M == -INFINITY ? 0.f : exp2_fast(M - top);
    // acc[cols c + e] of row n, register i: column 16 cols c + cols (4 g + i) + e
#pragma unroll
    for (int c = 0; c < S::kSets; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < S::kCols; e += 4)
          *reinterpret_cast<float4_t*>(&sums[wave][n][16 * S::kCols * c + S::kCols * (4 * g + i) + e]) =
              float4_t{acc[S::kCols * c + e][i] * f, acc[S::kCols * c + e + 1][i] * f, acc[S::kCols * c + e + 2][i] * f,
                       acc[S::kCols * c + e + 3][i] * f};
    __syncthreads();
    const bool complete = c0 == 0 && c1 == s.chunks;
    float* part = complete ? nullptr
                           : sp.parts + (2 * (int64_t)blockIdx.x + (c0 == 0 ? 1 : 0)) * (sp.part_rows * (D + 2));
    for (int i = tid; i < seg_rows * (D / 4); i += kThreads) {
      const int rr = i / (D / 4), d = 4 * (i - rr * (D / 4)), rn = rr % kRows, from = rr / kRows * streams;
      float best = stats[from][rn][0], sum = 0.f;
      for (int w = from + 1; w < from + streams; ++w) best = fmaxf(best, stats[w][rn][0]);
      float4_t o = float4_t{0.f, 0.f, 0.f, 0.f};
      for (int w = from; w < from + streams; ++w) {
        sum += stats[w][rn][0] == -INFINITY ? 0.f : stats[w][rn][1] * exp2_fast(stats[w][rn][0] - best);
        o += *reinterpret_cast<const float4_t*>(&sums[w][rn][d]);
      }
      if (complete) {
        const int grow = seg_row + rr, jj = grow / p.group;
        IO* out = static_cast<IO*>(p.output) + ((int64_t)(s.start + jj) * p.Hq + h * p.group + grow - jj * p.group) * D + d;
        const float norm = sum == 0.f ? 0.f : 1.f / sum;
        if constexpr (FMT == kF32)
          *reinterpret_cast<float4_t*>(out) = o * norm;
        else
          *reinterpret_cast<half4_t*>(out) = half4_t{(_Float16)(o[0] * norm), (_Float16)(o[1] * norm),
                                                     (_Float16)(o[2] * norm), (_Float16)(o[3] * norm)};
      } else {
        *reinterpret_cast<float4_t*>(part + 2 * sp.part_rows + rr * D + d) = o;
        if (d == 0) {
          part[rr] = best;
          part[sp.part_rows + rr] = sum;
        }
      }
    }
  }
}

// Joins the parts of the segments that several workgroups shared: a workgroup per
// (token, query head, 64 columns), its 16 slices of 16 lanes taking alternate parts.
// Parts are few and scattered, so latency counts: a slice loads several parts at once
// and joins them with a running M of its own.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) gdn_attn_join_k(AttnArgs p, SplitArgs sp, int groups) {
  typedef typename std::conditional<FMT == kF32, float, _Float16>::type IO;
  constexpr int kLanes = 16, kSlices = kThreads / kLanes, kSteps = D / 64, kAhead = 4;
  __shared__ float4_t sums[kSlices][kLanes];
  __shared__ float stats[kSlices][2];
  const int tid = threadIdx.x;
  const int id = (int)(blockIdx.x / kSteps), column = (int)(blockIdx.x % kSteps) * 64;
  const int n = id / p.Hq, head = id - n * p.Hq;
  const int64_t total = sp.prefix[p.rows.R];
  int r = 0;
  if (p.rows.cu_seqlens == nullptr) {
    r = n / p.rows.dense_len;
  } else {
    int hi = p.rows.R - 1;
    while (r < hi) {                                       // the first request that ends after n
      const int mid = (r + hi) >> 1;
      if (row_start(p.rows, mid + 1) <= n) r = mid + 1; else hi = mid;
    }
  }
  const Plan s = plan_of(p, r, sp.chunk_shift);
  if (n < s.start || n >= s.start + s.T) return;           // behind the last request
  const int h = head / p.group, row = (n - s.start) * p.group + head - h * p.group;
  const int seg = row / (kTiles * kRows), rr = row - seg * (kTiles * kRows);
  const int64_t share = share_of(total, groups);
  const int64_t from = sp.prefix[r] + ((int64_t)h * s.segs + seg) * s.chunks;
  const int64_t b0 = from / share;
  const int count = (int)((from + s.chunks - 1) / share - b0) + 1;
  if (count == 1) return;                                  // written by its one workgroup
  const int64_t size = (int64_t)sp.part_rows * (D + 2);
  const int slice = tid / kLanes, d = column + 4 * (tid - slice * kLanes);
  float4_t o = float4_t{0.f, 0.f, 0.f, 0.f};
  float M = -INFINITY, l = 0.f;
  for (int i = slice; i < count; i += kSlices * kAhead) {
    float m[kAhead], li[kAhead];
    float4_t x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // the first workgroup's part is its last segment, the others' their first; loads past
      // the last part repeat it
      const int at = min(i + k * kSlices, count - 1);
      const float* part = sp.parts + (2 * (b0 + at) + (at == 0 ? 1 : 0)) * size;
      m[k] = part[rr];
      li[k] = part[sp.part_rows + rr];
      x[k] = *reinterpret_cast<const float4_t*>(part + 2 * sp.part_rows + rr * D + d);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) top = i + k * kSlices < count ? fmaxf(top, m[k]) : top;
    const float f = M == -INFINITY ? 0.f : exp2_fast(M - top);
    o *= f;
    l *= f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float w = i + k * kSlices < count && m[k] != -INFINITY ? exp2_fast(m[k] - top) : 0.f;
      o += x[k] * w;
      l = fmaf(li[k], w, l);
    }
    M = top;
  }
  sums[slice][tid - slice * kLanes] = o;
  if (tid % kLanes == 0) {
    stats[slice][0] = M;
    stats[slice][1] = l;
  }
  __syncthreads();
  if (tid >= kLanes) return;
  float top = stats[0][0];
#pragma unroll
  for (int i = 1; i < kSlices; ++i) top = fmaxf(top, stats[i][0]);
  o = float4_t{0.f, 0.f, 0.f, 0.f};
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) {
    const float f = stats[i][0] == -INFINITY ? 0.f : exp2_fast(stats[i][0] - top);
    o += sums[i][tid] * f;
    l = fmaf(stats[i][1], f, l);
  }
  const float norm = l == 0.f ? 0.f : 1.f / l;
  IO* out = static_cast<IO*>(p.output) + ((int64_t)n * p.Hq + head) * D + d;
  if constexpr (FMT == kF32)
    *reinterpret_cast<float4_t*>(out) = o * norm;
  else
    *reinterpret_cast<half4_t*>(out) =
        half4_t{(_Float16)(o[0] * norm), (_Float16)(o[1] * norm), (_Float16)(o[2] * norm), (_Float16)(o[3] * norm)};
}

size_t prefix_bytes(int64_t R) { return ((size_t)(R + 1) * 8 + 255) & ~(size_t)255; }

// Rows of a part: a segment's, of at most kTiles tiles.
int part_rows(int64_t N, int group) {
  const int64_t tiles = (N * group + kRows - 1) / kRows;
  return (int)(tiles < kTiles ? tiles : kTiles) * kRows;
}

// Without a split a segment's positions pass through one workgroup, 128 at a time,
// and the second launch falls away.
constexpr int kWholeMax = 512;
constexpr int64_t kWholeGroups = 4096;

template <int FMT, int D>
hipError_t launch_attn_d(const AttnArgs& p, void* workspace, hipStream_t stream) {
  SplitArgs sp{};
  if (p.max_len <= kWholeMax) {
    sp.chunk_shift = kWholeShift;
    const int64_t segments = ((int64_t)p.rows.N * p.group / (kTiles * kRows) + p.rows.R) * p.cache.Hk;
    hipLaunchKernelGGL((gdn_attn_k<FMT, D>), dim3((unsigned)(segments < kWholeGroups ? segments : kWholeGroups)),
                       dim3(kThreads), 0, stream, p, sp);
    return hipGetLastError();
  }
  sp.prefix = static_cast<int64_t*>(workspace);
  sp.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + prefix_bytes(p.rows.R));
  sp.part_rows = part_rows(p.rows.N, p.group);
  sp.chunk_shift = kChunkShift;
  hipLaunchKernelGGL((gdn_attn_k<FMT, D>), dim3(kGroups), dim3(kThreads), 0, stream, p, sp);
  hipLaunchKernelGGL((gdn_attn_join_k<FMT, D>), dim3((unsigned)((int64_t)p.rows.N * p.Hq * (D / 64))), dim3(kThreads),
                     0, stream, p, sp, kGroups);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_attn_f(const AttnArgs& p, void* workspace, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_attn_d<FMT, 64>(p, workspace, stream);
    case 128: return launch_attn_d<FMT, 128>(p, workspace, stream);
    case 256: return launch_attn_d<FMT, 256>(p, workspace, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_attn(const AttnArgs& p, int io_dtype, void* workspace, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  if (io_dtype != 1) return launch_attn_f<kF32>(p, workspace, stream);
  return p.cache.e4m3 ? launch_attn_f<kE4M3>(p, workspace, stream) : launch_attn_f<kF16>(p, workspace, stream);
}

size_t attn_workspace_bytes(int64_t N, int64_t R, int Hq, int Hk, int D) {
  if (N == 0 || R == 0) return 0;
  return prefix_bytes(R) + (size_t)2 * kGroups * part_rows(N, Hq / Hk) * (D + 2) * sizeof(float);
}

}  // namespace gdn

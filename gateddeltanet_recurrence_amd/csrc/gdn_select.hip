// Selection of the pages that a token attends: gdn_kv_bounds and gdn_attn_select.
//
// A page's keys lie channel by channel within [low, high], so q . k over the page is at
// most sum_d max(q_d low_d, q_d high_d): for the heads that share a key head, w+ . high +
// w- . low with w+ (w-) the group's sum of the positive (negative) parts of q. That is two
// rows of D elements a page and head instead of page_size rows: the pages of the highest
// bounds are selected.
#include "gdn_attn_kernels.h"
#include "gdn_common.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Workgroups are numbered in the grid's x dimension, which takes 2^32 work-items.
constexpr int64_t kMostBlocks = (int64_t)1 << 23;

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
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

// 8 elements from element `at` of a cache row, as floats.
template <typename IO, int FMT, int D>
__device__ __forceinline__ void load_key8(const CacheArgs& c, int64_t row, int at, float (&x)[8]) {
  if constexpr (FMT == kCacheIo) {
    const IO* src = static_cast<const IO*>(c.k) + row * D + at;
    if constexpr (sizeof(IO) == 2) {
      const half8_t h = *reinterpret_cast<const half8_t*>(src);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (float)h[i];
    } else {
      const float4_t a = *reinterpret_cast<const float4_t*>(src), b = *reinterpret_cast<const float4_t*>(src + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
      }
    }
  } else if constexpr (FMT == kCacheE4M3) {
    const uint2_t w = *reinterpret_cast<const uint2_t*>(static_cast<const uint8_t*>(c.k) + row * D + at);
    const int s = c.k_scales[row];
    const float scale = __uint_as_float(s > 0 ? (uint32_t)s << 23 : 0x00400000u);   // 2^(s - 127)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      x[4 * i + 0] = lo[0] * scale;
      x[4 * i + 1] = lo[1] * scale;
      x[4 * i + 2] = hi[0] * scale;
      x[4 * i + 3] = hi[1] * scale;
    }
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.k) + row * (D / 2) + at / 2);
    const float scale = __uint_as_float((uint32_t)c.k_scales[block_scale_at(row, at >> 5, c.page_shift, D)] << 23);
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1];
    x[4] = d[0]; x[5] = d[1]; x[6] = e[0]; x[7] = e[1];
  }
}

// The lower (higher) of two, NaN where one is.
__device__ __forceinline__ float lower(float m, float x) { return x < m || x != x ? x : m; }
__device__ __forceinline__ float higher(float m, float x) { return x > m || x != x ? x : m; }

// A workgroup takes a head of the pages that begin within its tokens (a page is taken by
// its first token among a request's new ones): D / 8 lanes a key, 8 channels each.
template <typename IO, int D, int FMT>
__global__ void __launch_bounds__(kThreads) gdn_kv_bounds_k(BoundsArgs p) {
  constexpr int E = D / 8;                                 // lanes of a key
  constexpr int kAtOnce = kThreads / E;                    // keys of a step
  __shared__ float low[kWaves][D], high[kWaves][D];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ps = 1 << p.cache.page_shift;
  const int64_t work = ((int64_t)p.rows.N + p.tokens_per_block - 1) / p.tokens_per_block * p.cache.Hk;
  const int tokens = min(row_start(p.rows, p.rows.R), p.rows.N);
  for (int64_t job = blockIdx.x; job < work; job += gridDim.x) {
    const int h = (int)(job % p.cache.Hk), n0 = (int)(job / p.cache.Hk) * p.tokens_per_block;
    const int n1 = min(n0 + p.tokens_per_block, tokens);
    if (n0 >= n1) continue;
    int r = owner_of(p.rows, n0, lane);
    for (int n = n0; n < n1; ++n) {
      while (r + 1 < p.rows.R && row_start(p.rows, r + 1) <= n) ++r;
      const int64_t len = p.rows.seq_lens[r], pos = len - row_start(p.rows, r + 1) + n;
      if (n != row_start(p.rows, r) && (pos & (ps - 1)) != 0) continue;   // uniform: not the page's first
      const int64_t first = pos & ~(int64_t)(ps - 1), row = cache_row(p.cache, r, first);
      if (pos < 0 || row < 0) continue;
      const int64_t row0 = row + ((int64_t)h << p.cache.page_shift);
      const int count = (int)min((int64_t)ps, len - first), at = 8 * (tid % E);
      float lo[8], hi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = INFINITY;
        hi[i] = -INFINITY;
      }
      for (int k = tid / E; k < count; k += kAtOnce) {
        float x[8];
        load_key8<IO, FMT, D>(p.cache, row0 + k, at, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = lower(lo[i], x[i]);
          hi[i] = higher(hi[i], x[i]);
        }
      }
#pragma unroll
      for (int m = E; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = lower(lo[i], __shfl_xor(lo[i], m));
          hi[i] = higher(hi[i], __shfl_xor(hi[i], m));
        }
      if (lane < E) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          low[wave][at + i] = lo[i];
          high[wave][at + i] = hi[i];
        }
      }
      __syncthreads();
      IO* out = static_cast<IO*>(p.bounds) + (row0 >> p.cache.page_shift) * 2 * D;
      for (int i = tid; i < 2 * D; i += kThreads) {
        float m = i < D ? low[0][i] : high[0][i - D];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = i < D ? lower(m, low[w][i]) : higher(m, high[w][i - D]);
        out[i] = (IO)m;
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------- selection

// Scores are kept as 64-bit keys that order as they do: 0 for an entry that may not be
// selected, the highest for a NaN.
__device__ __forceinline__ uint64_t key_of(double x) {
  if (x != x) return ~(uint64_t)0;
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (b >> 63) != 0 ? ~b : b | ((uint64_t)1 << 63);
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// A token's pages: its request's table, the entries that it holds.
struct Token {
  const int32_t* table;
  int held;
};
__device__ __forceinline__ Token token_at(const SelectArgs& p, int n, int lane) {
  const int r = owner_of(p.rows, n, lane);
  const int64_t pos = (int64_t)p.rows.seq_lens[r] - row_start(p.rows, r + 1) + n;
  Token t;
  t.table = p.cache.table + (int64_t)r * p.cache.max_pages;
  t.held = pos < 0 ? 0 : (int)min((pos >> p.cache.page_shift) + 1, (int64_t)p.cache.max_pages);
  return t;
}

// 8 elements as doubles.
template <typename IO>
__device__ __forceinline__ void load8(const IO* src, double (&x)[8]) {
  if constexpr (sizeof(IO) == 2) {
    const half8_t h = *reinterpret_cast<const half8_t*>(src);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (double)(float)h[i];
  } else {
    const float4_t a = *reinterpret_cast<const float4_t*>(src), b = *reinterpret_cast<const float4_t*>(src + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = (double)a[i];
      x[4 + i] = (double)b[i];
    }
  }
}

// Keys of the entries [i0, i1) of token n, key head h: L = D / 16 lanes an entry, 16
// channels of both bounds each.
template <typename IO, int D>
__device__ __forceinline__ void score_entries(const SelectArgs& p, const Token& t, int n, int h, int i0, int i1, uint64_t* keys) {
  constexpr int L = D / 16;
  const int tid = threadIdx.x, e = tid % L;
  double plus[2][8], minus[2][8];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) plus[c][i] = minus[c][i] = 0.0;
  for (int g = 0; g < p.group; ++g) {
    const IO* q = static_cast<const IO*>(p.q) + (int64_t)n * p.q_stride + (int64_t)(h * p.group + g) * D;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      double x[8];
      load8(q + 8 * (c * L + e), x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        plus[c][i] += x[i] < 0.0 ? 0.0 : x[i];             // a NaN goes into both
        minus[c][i] += x[i] > 0.0 ? 0.0 : x[i];
      }
    }
  }
  for (int i = i0 + tid / L; i < i1; i += kThreads / L) {
    const int page = t.table[i];
    const bool there = page >= 0 && page < p.cache.num_pages;
    const IO* low = static_cast<const IO*>(p.bounds) + ((int64_t)(there ? page : 0) * p.cache.Hk + h) * 2 * D;
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      double lo[8], hi[8];
      load8(low + 8 * (c * L + e), lo);
      load8(low + D + 8 * (c * L + e), hi);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fma(plus[c][k], hi[k], fma(minus[c][k], lo[k], sum));
    }
    sum += dpp64<kDppQuadXor1>(sum);
    sum += dpp64<kDppQuadXor2>(sum);
    if constexpr (L >= 8) sum += dpp64<kDppHalfMirror>(sum);
    if constexpr (L >= 16) sum += dpp64<kDppRowMirror>(sum);
    if (e == 0) keys[i] = there ? key_of(sum) : 0;
  }
}

// Inclusive sum over a workgroup's threads, and the total. `sums` is free again after the call's second barrier.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t (&sums)[kWaves], uint64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t y = __shfl_up(x, m);
    if (lane >= m) x += y;
  }
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return x + before;
}

constexpr int kBuckets = 2048;

struct PickShared {
  uint32_t hist[kBuckets];
  uint64_t sums[kWaves], low[kWaves], high[kWaves];
  uint32_t bucket, above, inside;
};

// The K entries of a list from the keys of its `held` entries, those from `first_end` on and before `newest_begin`
// by key. The K-th largest key is found by counting keys in 2,048 equal parts of their range, and then in the part
// that it lies in, until every key of the part is taken or all are equal.
__device__ __forceinline__ void pick_entries(const SelectArgs& p, const uint64_t* keys, int held, int32_t* list, int32_t* count_out,
                                             PickShared& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, K = p.K;
  const int newest_begin = held - p.newest;
  uint64_t forced = 0, others = 0, lo = ~(uint64_t)0, hi = 0;
  for (int i = tid; i < held; i += kThreads) {
    const uint64_t key = keys[i];
    if (key == 0) continue;
    if (i < p.first || i >= newest_begin) {
      ++forced;
    } else {
      ++others;
      lo = min(lo, key);
      hi = max(hi, key);
    }
  }
  uint64_t both;
  block_scan(forced << 32 | others, s.sums, &both);
  const int64_t all_forced = (int64_t)(both >> 32), all_others = (int64_t)(both & 0xffffffffu);
  uint64_t over = 0;                                       // keys above this are taken, and `equal` of those that are it
  int64_t equal = 0;
  if (all_forced + all_others > K) {
    // the range of the others' keys
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      lo = min(lo, (uint64_t)__shfl_xor(lo, m));
      hi = max(hi, (uint64_t)__shfl_xor(hi, m));
    }
    if (lane == 0) {
      s.low[wave] = lo;
      s.high[wave] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      lo = min(lo, s.low[w]);
      hi = max(hi, s.high[w]);
    }
    int64_t need = K - all_forced;
    if (need <= 0) {
      over = ~(uint64_t)0;
    } else {
      for (;;) {
        const uint64_t range = hi - lo;
        const int bits = range == 0 ? 0 : 64 - __builtin_clzll(range), shift = max(bits - 11, 0);
        for (int i = tid; i < kBuckets; i += kThreads) s.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < held; i += kThreads) {
          const uint64_t key = keys[i];
          if (key >= lo && key <= hi && i >= p.first && i < newest_begin) atomicAdd(&s.hist[(key - lo) >> shift], 1u);
        }
        __syncthreads();
        // thread t holds buckets from the top: 8 t' .. 8 t' + 7, t' = 255 - t
        const int base = kBuckets / kThreads * (kThreads - 1 - tid);
        uint32_t mine[kBuckets / kThreads];
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kBuckets / kThreads; ++i) {
          mine[i] = s.hist[base + i];
          sum += mine[i];
        }
        uint64_t total;
        const uint64_t upto = block_scan(sum, s.sums, &total);
        if ((int64_t)(upto - sum) < need && need <= (int64_t)upto) {
          uint64_t above = upto - sum;
          int b = kBuckets / kThreads - 1;
#pragma unroll
          for (int i = kBuckets / kThreads - 1; i > 0; --i)
            if (b == i && (int64_t)(above + mine[i]) < need) {
              above += mine[i];
              b = i - 1;
            }
          s.bucket = (uint32_t)(base + b);
          s.above = (uint32_t)above;
          s.inside = 0;
#pragma unroll
          for (int i = 0; i < kBuckets / kThreads; ++i)
            if (b == i) s.inside = mine[i];
        }
        __syncthreads();
        need -= s.above;
        lo += (uint64_t)s.bucket << shift;
        hi = min(hi, lo + (((uint64_t)1 << shift) - 1));
        const bool done = (int64_t)s.inside == need, same = shift == 0;
        __syncthreads();                                   // s is written again
        if (done || same) {
          over = done ? lo - 1 : lo;
          equal = done ? 0 : need;
          break;
        }
      }
    }
  }
  // in order: each thread's entries are neighbours
  const int per = (held + kThreads - 1) / kThreads, i0 = min(tid * per, held), i1 = min(i0 + per, held);
  uint64_t taken = 0, ties = 0;
  for (int i = i0; i < i1; ++i) {
    const uint64_t key = keys[i];
    const bool always = key != 0 && (i < p.first || i >= newest_begin);
    taken += always || key > over ? 1 : 0;
    ties += !always && key != 0 && key == over ? 1 : 0;
  }
  uint64_t total;
  const uint64_t upto = block_scan(taken << 32 | ties, s.sums, &total);
  int64_t ties_before = (int64_t)(upto & 0xffffffffu) - (int64_t)ties;
  int64_t at = (int64_t)(upto >> 32) - (int64_t)taken + min(ties_before, equal);
  for (int i = i0; i < i1; ++i) {
    const uint64_t key = keys[i];
    const bool always = key != 0 && (i < p.first || i >= newest_begin), tie = !always && key != 0 && key == over;
    if (always || key > over || (tie && ties_before < equal)) list[at++] = i;
    if (tie) ++ties_before;
  }
  const int count = (int)((int64_t)(total >> 32) + min((int64_t)(total & 0xffffffffu), equal));
  for (int i = count + tid; i < K; i += kThreads) list[i] = -1;
  if (tid == 0 && count_out != nullptr) *count_out = count;
}

// One list a workgroup: all of its keys, then the selection among them.
template <typename IO, int D>
__global__ void __launch_bounds__(kThreads) gdn_attn_select_k(SelectArgs p) {
  __shared__ PickShared shared;
  const int64_t lists = (int64_t)min(row_start(p.rows, p.rows.R), p.rows.N) * p.cache.Hk;
  for (int64_t job = blockIdx.x; job < lists; job += gridDim.x) {
    const int n = (int)(job / p.cache.Hk), h = (int)(job % p.cache.Hk);
    const Token t = token_at(p, n, threadIdx.x & 63);
    uint64_t* keys = p.keys + job * p.cache.max_pages;
    score_entries<IO, D>(p, t, n, h, 0, t.held, keys);
    __syncthreads();
    pick_entries(p, keys, t.held, p.pages + job * p.K, h == 0 ? p.counts + n : nullptr, shared);
    __syncthreads();
  }
}

template <typename IO, int D>
hipError_t launch_bounds_d(const BoundsArgs& p, hipStream_t stream) {
  const int64_t jobs = ((int64_t)p.rows.N + p.tokens_per_block - 1) / p.tokens_per_block * p.cache.Hk;
  const dim3 grid((unsigned)(jobs < kMostBlocks ? jobs : kMostBlocks));
  if (p.cache.format == kCacheIo) {
    hipLaunchKernelGGL((gdn_kv_bounds_k<IO, D, kCacheIo>), grid, dim3(kThreads), 0, stream, p);
  } else {
    if constexpr (sizeof(IO) == 2) {
      if (p.cache.format == kCacheE4M3)
        hipLaunchKernelGGL((gdn_kv_bounds_k<IO, D, kCacheE4M3>), grid, dim3(kThreads), 0, stream, p);
      else
        hipLaunchKernelGGL((gdn_kv_bounds_k<IO, D, kCacheE2M1>), grid, dim3(kThreads), 0, stream, p);
    } else {
      return hipErrorInvalidValue;
    }
  }
  return hipGetLastError();
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

template <typename IO, int D>
hipError_t launch_select_d(const SelectArgs& p, hipStream_t stream) {
  const int64_t lists = (int64_t)p.rows.N * p.cache.Hk;
  const dim3 grid((unsigned)(lists < kMostBlocks ? lists : kMostBlocks));
  hipLaunchKernelGGL((gdn_attn_select_k<IO, D>), grid, dim3(kThreads), 0, stream, p);
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

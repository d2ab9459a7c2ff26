// Rotary positions and the paged key-value cache: gdn_rope_forward,
// gdn_kv_write, gdn_kv_read.
//
// All three move every element once and compute a handful of operations on it,
// so they are bound by HBM for prompts and by latency for a decode step. A
// thread handles 2 x 16 bytes of one head of one token (an "item"): for a
// rotated item the two vectors hold the partners of 8 (fp16) or 4 (fp32) pairs
// in the half layout, and in both layouts the lanes of an item row touch
// consecutive 16-byte vectors. A workgroup takes a few whole tokens, forms the
// cos and sin of each of their pairs once into LDS (shared by all heads), finds
// where each token lives in the cache, and then walks the tokens' heads: q
// heads, k heads and, for the cache write, v heads.
#include "gdn_attn_kernels.h"
#include "gdn_common.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// A launch has fewer than 2^32 work-items in a dimension (more are dropped without an error): workgroups past 2^23
// go to the second one. The first token of this workgroup, at most N.
constexpr int kGridShift = 23;
dim3 grid_of(int64_t N, int tokens_per_block) {
  const int64_t blocks = (N + tokens_per_block - 1) / tokens_per_block, wide = (int64_t)1 << kGridShift;
  return dim3((unsigned)(blocks < wide ? blocks : wide), (unsigned)((blocks + wide - 1) >> kGridShift));
}
__device__ __forceinline__ int first_token(int N, int tokens_per_block) {
  const unsigned n0 = ((blockIdx.y << kGridShift) + blockIdx.x) * (unsigned)tokens_per_block;   // below 2^31 + 2^27
  return (int)min(n0, (unsigned)N);
}

// A 16-byte vector of io elements.
template <typename IO> struct Vec;
template <> struct Vec<_Float16> {
  static constexpr int n = 8;
  typedef half8_t type;
};
template <> struct Vec<float> {
  static constexpr int n = 4;
  typedef float4_t type;
};

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));

// Outputs are written once and not read here: nontemporal stores (32,768 tokens read
// back 39 -> 31 us, 15,352 written in 8 bits 36 -> 30 us). Nontemporal loads of the
// inputs were slower (31 -> 38 us, 30 -> 35 us): two loads share a 128-byte line.
template <typename T, typename P> __device__ __forceinline__ void store_stream(P* p, T x) {
  __builtin_nontemporal_store(x, reinterpret_cast<T*>(p));
}

// Largest of x over aligned groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ float group_max(float x) {
  static_assert(LANES == 4 || LANES == 8 || LANES == 16, "group of 4, 8 or 16 lanes");
  x = fmaxf(x, dpp<kDppQuadXor1>(x));
  x = fmaxf(x, dpp<kDppQuadXor2>(x));
  if constexpr (LANES >= 8) x = fmaxf(x, dpp<kDppHalfMirror>(x));
  if constexpr (LANES >= 16) x = fmaxf(x, dpp<kDppRowMirror>(x));
  return x;
}

// Exponent byte s of a row with largest finite magnitude a: 2^(s - 127) is the
// smallest power of two with a <= 448 * 2^(s - 127). With a = 1.m * 2^e and
// 448 = 1.75 * 2^8 that is 2^(e - 8), or twice it when 1.m > 1.75. fp16 values
// are normal floats, so e is the exponent field and s lies in 95 .. 135.
__device__ __forceinline__ int scale_byte(float a) {
  const uint32_t b = __float_as_uint(a);
  return a > 0.f ? (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0) : 0;
}

__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// e4m3 codes of 8 values times inv (a power of two, so the products are exact);
// v_cvt_pk_fp8_f32 rounds to nearest even.
__device__ __forceinline__ uint2_t encode8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = is_finite(x[i]) ? x[i] * inv : __uint_as_float(0x7fc00000u);
  int a = 0, b = 0;
  a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], a, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], b, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
  return uint2_t{(uint32_t)a, (uint32_t)b};
}

// Exponent byte of a block of 32 whose largest magnitude has the fp16 bits `bits`: 2^(s - 127) is the smallest power
// of two, up to 2^13, with a <= 6 * 2^(s - 127). With a = 1.m * 2^e and 6 = 1.5 * 2^2 that is 2^(e - 2), or twice it
// when 1.m > 1.5; 255 for an infinity or NaN.
__device__ __forceinline__ int block_scale_byte(uint32_t bits) {
  if (bits >= 0x7c00u) return 255;
  const uint32_t b = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)bits));
  return bits > 0 ? min((int)(b >> 23) - 2 + ((b & 0x7fffffu) > 0x400000u ? 1 : 0), 140) : 0;
}

// Magnitude bits of two halves, the larger of each half.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t a, uint32_t b) {
  typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a & 0x7fff7fffu),
                                                                __builtin_bit_cast(ushort2_t, b & 0x7fff7fffu)));
}

// e2m1 codes of 8 halves over the scale: v_cvt_scalef32_pk_fp4_f16 divides exactly, rounds to nearest even and stops at 6.
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t encode4(const uint32_t (&w)[4], float scale) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[0]), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[1]), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[2]), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(half2_t, w[3]), scale, 3);
  return c;
}

// 8 e2m1 codes times 2^(s - 127), exact (s = 255: NaN).
__device__ __forceinline__ half8_t decode4(uint32_t c, int s) {
  const float scale = __uint_as_float((uint32_t)s << 23);
  typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(half8_t, uint4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 0)),
                                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 1)),
                                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 2)),
                                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 3))});
}

// Request of the workgroup's first token n0 (the same in every thread): the
// number of requests that end at or before n0, at most R - 1. Every thread must
// call it; the result lies in [0, R) whatever cu_seqlens holds.
__device__ __forceinline__ int request_of(const RowArgs& p, int n0) {
  if (p.cu_seqlens == nullptr) return min(n0 / p.dense_len, p.R - 1);
  __shared__ int counts[kThreads / 64];
  int mine = 0;
  for (int i = threadIdx.x; i < p.R; i += kThreads) mine += row_start(p, i + 1) <= n0 ? 1 : 0;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) mine += __shfl_xor(mine, m);
  if ((threadIdx.x & 63) == 0) counts[threadIdx.x >> 6] = mine;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) all += counts[w];
  return min(all, p.R - 1);
}

// Tokens of the call that belong to a request: those behind the last one
// (cu_seqlens[R] < N, a padded batch) are left as they are.
__device__ __forceinline__ int row_count(const RowArgs& p) { return min(row_start(p, p.R), p.N); }

// Position of token n < row_count of request r or a later one (r is advanced to
// the first that ends after n): seq_lens[r] - T_r + j.
__device__ __forceinline__ int64_t position_of(const RowArgs& p, int n, int& r) {
  if (p.cu_seqlens == nullptr) {
    r = min(n / p.dense_len, p.R - 1);
  } else {
    while (r + 1 < p.R && row_start(p, r + 1) <= n) ++r;
  }
  return (int64_t)p.seq_lens[r] - row_start(p, r + 1) + n;
}

// factor cos t and factor sin t of t = position * frequency, rounded once to float wherever the position lies: the
// product and its share of a turn are kept as sums of two doubles, so that what is left of the angle, y, at most an
// eighth of a turn, has all its digits (one double holds a far position's angle only to 2^-52 of it: 2^-21 at 2^31).
// The power series' terms up to y^13 and y^12 leave less than 2^-40.
__device__ __forceinline__ float2 turn_of(double position, double frequency, double factor) {
  constexpr double kInvTwoPi = 0.15915494309189533577, kInvTwoPiLow = -9.839338337591243e-18;
  constexpr double kTwoPi = 6.283185307179586477;
  const double t = position * frequency, turn = t * kInvTwoPi, quarter = rint(4.0 * turn);
  const double low = fma(t, kInvTwoPi, -turn) + fma(fma(position, frequency, -t), kInvTwoPi, t * kInvTwoPiLow);
  const double y = (fma(-0.25, quarter, turn) + low) * kTwoPi, z = y * y;
  double s = 1.0 / 6227020800.0, c = 1.0 / 479001600.0;    // 1 / 13!, 1 / 12!
  s = fma(s, z, -1.0 / 39916800.0);
  c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, 1.0 / 362880.0);
  c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, -1.0 / 5040.0);
  c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, 1.0 / 120.0);
  c = fma(c, z, 1.0 / 24.0);
  s = fma(s, z, -1.0 / 6.0);
  c = fma(c, z, -0.5);
  s = fma(s * z, y, y) * factor;
  c = fma(c, z, 1.0) * factor;
  const int q = (int)(quarter - 4.0 * floor(0.25 * quarter));
  const float fs = (float)s, fc = (float)c;
  const float a = q & 1 ? fs : fc, b = q & 1 ? fc : fs;    // cos, sin after q quarter turns
  return float2{q == 1 || q == 2 ? -a : a, q >= 2 ? -b : b};
}

template <typename IO, int D, bool CACHE, int FMT>
__global__ void __launch_bounds__(kThreads) gdn_rope_k(RopeArgs p) {
  constexpr int V = Vec<IO>::n;            // elements of a vector
  constexpr int E = D / (2 * V);           // items of a head
  constexpr int kHeadStep = kThreads / E;
  typedef typename Vec<IO>::type vec_t;
  __shared__ int64_t row_of[kRopeMaxTokens];
  __shared__ double pos_of[kRopeMaxTokens];
  extern __shared__ float2 turns[];        // [tokens][rot / 2] cos and sin

  const int n0 = first_token(p.N, p.tokens_per_block);
  const int tokens = min(p.tokens_per_block, (CACHE ? row_count(p.rows) : p.N) - n0);
  if (tokens <= 0) return;                 // uniform across the workgroup
  const int pairs = p.rot >> 1;
  if constexpr (CACHE) {
    int r = request_of(p.rows, n0);
    if ((int)threadIdx.x < tokens) {
      const int n = n0 + threadIdx.x;
      const int64_t pos = position_of(p.rows, n, r);
      row_of[threadIdx.x] = cache_row(p.cache, r, pos);
      pos_of[threadIdx.x] = p.positions != nullptr ? (double)p.positions[n] : (double)pos;
    }
  } else {
    if ((int)threadIdx.x < tokens) pos_of[threadIdx.x] = (double)p.positions[n0 + threadIdx.x];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs;
    turns[i] = turn_of(pos_of[t], p.inv_freq[i - t * pairs], (double)p.factor);
  }
  __syncthreads();

  const int e = threadIdx.x % E;
  const bool rotated = e < p.rot / (2 * V);
  // the item's vectors lie at a and b of the head
  const int base = rotated ? 0 : p.rot, size = rotated ? p.rot : D - p.rot;
  const int a = base + V * (rotated ? e : e - p.rot / (2 * V)), b = a + (size >> 1);
  const int heads = p.Hq + p.Hk + (CACHE ? p.Hk : 0);

  int t = 0, h = threadIdx.x / E;
  for (;; h += kHeadStep) {
    while (h >= heads) {
      h -= heads;
      ++t;
    }
    if (t >= tokens) break;
    const int64_t n = n0 + t;
    const bool is_q = h < p.Hq, is_v = CACHE && h >= p.Hq + p.Hk;
    const int hh = is_q ? h : is_v ? h - p.Hq - p.Hk : h - p.Hq;
    const IO* src = is_q ? static_cast<const IO*>(p.q) + n * p.q_stride
                         : is_v ? static_cast<const IO*>(p.v) + n * p.v_stride
                                : static_cast<const IO*>(p.k) + n * p.k_stride;
    src += hh * D;
    const bool turn = rotated && !is_v;
    const bool keep = !turn && (is_q ? p.q_in_place : !CACHE && p.k_in_place);   // in place, not rotated
    float x[V], y[V];
    if (!keep) {
      const vec_t xa = *reinterpret_cast<const vec_t*>(src + a), xb = *reinterpret_cast<const vec_t*>(src + b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = (float)xa[i];
        y[i] = (float)xb[i];
      }
    }
    if (turn) {
      const float2* cs = turns + t * pairs;
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 ta = cs[(a + i) >> 1], tb = cs[(b + i) >> 1];
          const float x0 = x[i], x1 = x[i + 1], y0 = y[i], y1 = y[i + 1];
          x[i] = x0 * ta.x - x1 * ta.y;
          x[i + 1] = x1 * ta.x + x0 * ta.y;
          y[i] = y0 * tb.x - y1 * tb.y;
          y[i + 1] = y1 * tb.x + y0 * tb.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 ti = cs[a + i];
          const float xi = x[i], yi = y[i];
          x[i] = xi * ti.x - yi * ti.y;
          y[i] = yi * ti.x + xi * ti.y;
        }
      }
    }
    vec_t ra, rb;
    if (!keep) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ra[i] = (IO)x[i];
        rb[i] = (IO)y[i];
      }
    }
    if (is_q || !CACHE) {
      if (keep) continue;
      IO* dst = (is_q ? static_cast<IO*>(p.q_out) + n * p.q_out_stride
                      : static_cast<IO*>(p.k_out) + n * p.k_out_stride) + hh * D;
      store_stream(dst + a, ra);
      store_stream(dst + b, rb);
      continue;
    }
    if constexpr (CACHE) {
      // the lanes of a head share its token, so they leave together
      if (row_of[t] < 0) continue;
      const int64_t row = row_of[t] + ((int64_t)hh << p.cache.page_shift);
      if constexpr (FMT == kCacheE4M3) {
        // what is stored is the io value's code, as if k had been rotated and written apart
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[i] = (float)ra[i];
          y[i] = (float)rb[i];
          if (is_finite(x[i])) m = fmaxf(m, fabsf(x[i]));
          if (is_finite(y[i])) m = fmaxf(m, fabsf(y[i]));
        }
        m = group_max<E>(m);
        const int s = scale_byte(m);
        const float inv = __uint_as_float((uint32_t)(s > 0 ? 254 - s : 127) << 23);
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k) + row * D;
        store_stream(dst + a, encode8(x, inv));
        store_stream(dst + b, encode8(y, inv));
        if (e == 0) (is_v ? p.cache.v_scales : p.cache.k_scales)[row] = (uint8_t)s;
      } else if constexpr (FMT == kCacheE2M1) {
        // Blocks of 32 neighbours: the halves of a rotation lie in other lanes, so a head's row goes through LDS and
        // comes back 16 elements a lane. Its lanes are of one wave, whose LDS accesses keep their order.
        __shared__ alignas(16) _Float16 heads_row[kThreads / E][D];
        typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
        _Float16* mine = heads_row[threadIdx.x / E];
        *reinterpret_cast<vec_t*>(mine + a) = ra;
        *reinterpret_cast<vec_t*>(mine + b) = rb;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const uint4_t lo4 = *reinterpret_cast<const uint4_t*>(mine + 16 * e), hi4 = *reinterpret_cast<const uint4_t*>(mine + 16 * e + 8);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const uint32_t lo[4] = {lo4[0], lo4[1], lo4[2], lo4[3]}, hi[4] = {hi4[0], hi4[1], hi4[2], hi4[3]};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_magnitudes(m, max_magnitudes(lo[i], hi[i]));
        m = max(m & 0xffffu, m >> 16);
        m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor1, 0xF, 0xF, true));
        const int s = block_scale_byte(m);
        const float scale = __uint_as_float((uint32_t)(s == 0 || s == 255 ? 127 : s) << 23);
        uint2_t codes = uint2_t{encode4(lo, scale), encode4(hi, scale)};
        if (s == 255) codes = uint2_t{0, 0};
        store_stream(static_cast<uint8_t*>(is_v ? p.cache.v : p.cache.k) + row * (D / 2) + 8 * e, codes);
        if ((e & 1) == 0)
          (is_v ? p.cache.v_scales : p.cache.k_scales)[block_scale_at(row, e >> 1, p.cache.page_shift, D)] = (uint8_t)s;
      } else {
        IO* dst = static_cast<IO*>(is_v ? p.cache.v : p.cache.k) + row * D;
        store_stream(dst + a, ra);
        store_stream(dst + b, rb);
      }
    }
  }
}

template <typename IO, int D, int FMT>
__global__ void __launch_bounds__(kThreads) gdn_kv_read_k(ReadArgs p) {
  constexpr int V = Vec<IO>::n;
  constexpr int E = D / (2 * V);
  constexpr int kHeadStep = kThreads / E;
  typedef typename Vec<IO>::type vec_t;
  __shared__ int64_t row_of[kRopeMaxTokens];
  const int n0 = first_token(p.rows.N, p.tokens_per_block);
  const int tokens = min(p.tokens_per_block, row_count(p.rows) - n0);
  if (tokens <= 0) return;
  int r = request_of(p.rows, n0);
  if ((int)threadIdx.x < tokens) {
    const int64_t pos = position_of(p.rows, n0 + threadIdx.x, r);
    row_of[threadIdx.x] = cache_row(p.cache, r, pos);
  }
  __syncthreads();
  const int a = V * (threadIdx.x % E), b = a + D / 2;
  const int Hk = p.cache.Hk, heads = 2 * Hk;
  int t = 0, h = threadIdx.x / E;
  for (;; h += kHeadStep) {
    while (h >= heads) {
      h -= heads;
      ++t;
    }
    if (t >= tokens) break;
    const bool is_v = h >= Hk;
    const int hh = is_v ? h - Hk : h;
    vec_t xa = {}, xb = {};
    if (row_of[t] >= 0) {
      const int64_t row = row_of[t] + ((int64_t)hh << p.cache.page_shift);
      if constexpr (FMT == kCacheE4M3) {
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.cache.v : p.cache.k) + row * D;
        const uint2_t ca = *reinterpret_cast<const uint2_t*>(src + a), cb = *reinterpret_cast<const uint2_t*>(src + b);
        const int s = (is_v ? p.cache.v_scales : p.cache.k_scales)[row];
        const float scale = __uint_as_float(s > 0 ? (uint32_t)s << 23 : 0x00400000u);   // 2^(s - 127)
        const uint32_t w[4] = {ca.x, ca.y, cb.x, cb.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
          const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
          vec_t& to = i < 2 ? xa : xb;
          to[4 * (i & 1) + 0] = (IO)(lo[0] * scale);
          to[4 * (i & 1) + 1] = (IO)(lo[1] * scale);
          to[4 * (i & 1) + 2] = (IO)(hi[0] * scale);
          to[4 * (i & 1) + 3] = (IO)(hi[1] * scale);
        }
      } else if constexpr (FMT == kCacheE2M1) {
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.cache.v : p.cache.k) + row * (D / 2);
        const uint8_t* scales = is_v ? p.cache.v_scales : p.cache.k_scales;
        xa = decode4(*reinterpret_cast<const uint32_t*>(src + a / 2), scales[block_scale_at(row, a >> 5, p.cache.page_shift, D)]);
        xb = decode4(*reinterpret_cast<const uint32_t*>(src + b / 2), scales[block_scale_at(row, b >> 5, p.cache.page_shift, D)]);
      } else {
        const IO* src = static_cast<const IO*>(is_v ? p.cache.v : p.cache.k) + row * D;
        xa = *reinterpret_cast<const vec_t*>(src + a);
        xb = *reinterpret_cast<const vec_t*>(src + b);
      }
    }
    IO* dst = static_cast<IO*>(is_v ? p.v : p.k) + ((int64_t)(n0 + t) * Hk + hh) * D;
    store_stream(dst + a, xa);
    store_stream(dst + b, xb);
  }
}

template <typename IO, int D>
hipError_t launch_rope_d(const RopeArgs& p, hipStream_t stream) {
  const dim3 grid = grid_of(p.N, p.tokens_per_block);
  const size_t lds = (size_t)p.tokens_per_block * (p.rot / 2) * sizeof(float2);
  if (!p.to_cache) {
    hipLaunchKernelGGL((gdn_rope_k<IO, D, false, kCacheIo>), grid, dim3(kThreads), lds, stream, p);
  } else if (p.cache.format == kCacheIo) {
    hipLaunchKernelGGL((gdn_rope_k<IO, D, true, kCacheIo>), grid, dim3(kThreads), lds, stream, p);
  } else {
    if constexpr (sizeof(IO) == 2) {
      if (p.cache.format == kCacheE4M3)
        hipLaunchKernelGGL((gdn_rope_k<IO, D, true, kCacheE4M3>), grid, dim3(kThreads), lds, stream, p);
      else
        hipLaunchKernelGGL((gdn_rope_k<IO, D, true, kCacheE2M1>), grid, dim3(kThreads), lds, stream, p);
    } else {
      return hipErrorInvalidValue;
    }
  }
  return hipGetLastError();
}

template <typename IO, int D>
hipError_t launch_read_d(const ReadArgs& p, hipStream_t stream) {
  const dim3 grid = grid_of(p.rows.N, p.tokens_per_block);
  if (p.cache.format == kCacheIo) {
    hipLaunchKernelGGL((gdn_kv_read_k<IO, D, kCacheIo>), grid, dim3(kThreads), 0, stream, p);
  } else {
    if constexpr (sizeof(IO) == 2) {
      if (p.cache.format == kCacheE4M3)
        hipLaunchKernelGGL((gdn_kv_read_k<IO, D, kCacheE4M3>), grid, dim3(kThreads), 0, stream, p);
      else
        hipLaunchKernelGGL((gdn_kv_read_k<IO, D, kCacheE2M1>), grid, dim3(kThreads), 0, stream, p);
    } else {
      return hipErrorInvalidValue;
    }
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_rope_io(const RopeArgs& p, hipStream_t stream) {
  switch (p.D) {
    case 64: return launch_rope_d<IO, 64>(p, stream);
    case 128: return launch_rope_d<IO, 128>(p, stream);
    case 256: return launch_rope_d<IO, 256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

template <typename IO>
hipError_t launch_read_io(const ReadArgs& p, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_read_d<IO, 64>(p, stream);
    case 128: return launch_read_d<IO, 128>(p, stream);
    case 256: return launch_read_d<IO, 256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& p, int io_dtype, hipStream_t stream) {
  if (p.N == 0) return hipSuccess;
  return io_dtype == 1 ? launch_rope_io<_Float16>(p, stream) : launch_rope_io<float>(p, stream);
}

hipError_t launch_kv_read(const ReadArgs& p, int io_dtype, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  return io_dtype == 1 ? launch_read_io<_Float16>(p, stream) : launch_read_io<float>(p, stream);
}

}  // namespace gdn

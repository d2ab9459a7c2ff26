// Attention of every request's newest tokens over its paged cache:
// gdn_attn_forward.
//
// One wave per (token, query head) walks the attended positions one by one with
// the running maximum m and sum l of the softmax:
//   s = scale q.k;  m' = max(m, s);  c = e^(m - m');  w = e^(s - m')
//   l = c l + w;  o = c o + w v
// in FP32, the head's D elements spread over the lanes.
#include "gdn_attn_kernels.h"
#include "gdn_common.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

template <typename IO, int D, bool E4M3>
__device__ __forceinline__ void load_row(const void* pages, const uint8_t* scales, int64_t row, int lane,
                                         float (&x)[D / 64]) {
  if constexpr (E4M3) {
    const int s = scales[row];
    const float scale = __uint_as_float(s > 0 ? (uint32_t)s << 23 : 0x00400000u);
    const uint8_t* src = static_cast<const uint8_t*>(pages) + row * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) x[i] = __builtin_amdgcn_cvt_f32_fp8((int)src[lane + 64 * i], 0) * scale;
  } else {
    const IO* src = static_cast<const IO*>(pages) + row * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) x[i] = (float)src[lane + 64 * i];
  }
}

template <typename IO, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) gdn_attn_simple_k(AttnArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t id = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
  if (id >= (int64_t)p.rows.N * p.Hq) return;
  const int n = (int)(id / p.Hq), h = (int)(id % p.Hq);
  int lo = 0, hi = p.rows.R - 1;                 // the first request that ends after n
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (row_start(p.rows, mid + 1) <= n) lo = mid + 1; else hi = mid;
  }
  const int r = lo;
  if (n >= row_start(p.rows, p.rows.R)) return;  // behind the last request: left as it is
  const int64_t last = (int64_t)p.rows.seq_lens[r] - row_start(p.rows, r + 1) + n;
  const int64_t cap = (int64_t)p.cache.max_pages << p.cache.page_shift;
  const int64_t end = last + 1 < cap ? last + 1 : cap;
  int64_t begin = p.window > 0 ? last - p.window + 1 : 0;
  if (begin < 0) begin = 0;
  constexpr int E = D / 64;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const IO* qs = static_cast<const IO*>(p.q) + (int64_t)n * p.q_stride + h * D;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = (float)qs[lane + 64 * i];
    o[i] = 0.f;
  }
  const int64_t head = (int64_t)(h / p.group) << p.cache.page_shift;
  for (int64_t pos = begin; pos < end; ++pos) {
    const int64_t row = cache_row(p.cache, r, pos);
    if (row < 0) continue;
    float x[E], s = 0.f;
    load_row<IO, D, E4M3>(p.cache.k, p.cache.k_scales, row + head, lane, x);
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    s *= p.scale;
    const float m2 = fmaxf(m, s);
    const float c = m2 > m ? expf(m - m2) : 1.f, w = expf(s - m2);
    load_row<IO, D, E4M3>(p.cache.v, p.cache.v_scales, row + head, lane, x);
    l = l * c + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(w, x[i], o[i] * c);
    m = m2;
  }
  IO* out = static_cast<IO*>(p.output) + ((int64_t)n * p.Hq + h) * D;
#pragma unroll
  for (int i = 0; i < E; ++i) out[lane + 64 * i] = (IO)(l == 0.f ? 0.f : o[i] / l);
}

template <typename IO, int D>
hipError_t launch_attn_d(const AttnArgs& p, hipStream_t stream) {
  const int64_t waves = (int64_t)p.rows.N * p.Hq;
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (!p.cache.e4m3) {
    hipLaunchKernelGGL((gdn_attn_simple_k<IO, D, false>), grid, dim3(kThreads), 0, stream, p);
  } else {
    if constexpr (sizeof(IO) == 2)
      hipLaunchKernelGGL((gdn_attn_simple_k<IO, D, true>), grid, dim3(kThreads), 0, stream, p);
    else
      return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_attn_io(const AttnArgs& p, hipStream_t stream) {
  switch (p.cache.D) {
    case 64: return launch_attn_d<IO, 64>(p, stream);
    case 128: return launch_attn_d<IO, 128>(p, stream);
    case 256: return launch_attn_d<IO, 256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_attn(const AttnArgs& p, int io_dtype, void* workspace, hipStream_t stream) {
  (void)workspace;
  if (p.rows.N == 0) return hipSuccess;
  return io_dtype == 1 ? launch_attn_io<_Float16>(p, stream) : launch_attn_io<float>(p, stream);
}

size_t attn_workspace_bytes(int64_t N, int64_t R, int Hq, int Hk, int D) {
  (void)N; (void)R; (void)Hq; (void)Hk; (void)D;
  return 0;
}

}  // namespace gdn

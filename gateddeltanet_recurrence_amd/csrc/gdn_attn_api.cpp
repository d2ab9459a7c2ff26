// C ABI of the attention layer's serving step (gdn_attn.h): argument
// validation and dispatch. As in gdn_api.cpp every check runs on the host
// before any launch, so an error status other than GDN_ERR_HIP leaves device
// memory untouched.
#include "../../include/gdn_attn.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <new>
#include <utility>

#include "gdn_attn_kernels.h"
#include "gdn_host.h"

namespace {

using gdn::Span;
using gdn::aligned16;
using gdn::io_bytes;

constexpr double kPi = 3.14159265358979323846;
constexpr int64_t kMaxPositions = (int64_t)1 << 30;

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_size_ok(int s) { return s >= 16 && s <= 1024 && (s & (s - 1)) == 0; }

// `count` rows of `width` bytes, `stride` bytes apart (stride >= width).
struct RowSpan {
  uintptr_t lo = 0;
  size_t width = 0, stride = 0, count = 0;
  RowSpan() = default;
  RowSpan(const void* p, size_t w, size_t s, size_t n)
      : lo(reinterpret_cast<uintptr_t>(p)), width(w), stride(s), count(p == nullptr || w == 0 ? 0 : n) {}
  Span all() const {
    Span x;
    if (count > 0) {
      x.lo = lo;
      x.hi = lo + (count - 1) * stride + width;
    }
    return x;
  }
  // Rows of one stride interleave without touching when each set stays within
  // the other's gaps: q, k and v side by side in one buffer.
  bool overlaps(const RowSpan& o) const {
    if (!all().overlaps(o.all())) return false;
    if (stride != o.stride) return true;
    const size_t d = lo <= o.lo ? (o.lo - lo) % stride : (stride - (lo - o.lo) % stride) % stride;
    return !(d >= width && d + o.width <= stride);
  }
  bool overlaps(const Span& s) const { return all().overlaps(s); }
};

// A token stride as given (0: dense) in elements, or -1 where it is out of range.
int64_t token_stride(int32_t given, int64_t heads, int64_t D) {
  if (given == 0) return heads * D;
  return given >= heads * D && given % 8 == 0 ? given : -1;
}

int check_cache(const gdn_kv_cache* c, bool pointers) {
  if (c == nullptr) return GDN_ERR_NULL;
  if (c->io_dtype != GDN_F32 && c->io_dtype != GDN_F16) return GDN_ERR_DTYPE;
  if (c->format != GDN_CACHE_IO && c->format != GDN_CACHE_E4M3) return GDN_ERR_DTYPE;
  if (c->format == GDN_CACHE_E4M3 && c->io_dtype != GDN_F16) return GDN_ERR_DTYPE;
  if (c->num_pages < 1 || c->max_pages < 1 || c->num_kv_heads < 1) return GDN_ERR_SHAPE;
  if (!page_size_ok(c->page_size) || !head_dim_ok(c->head_dim)) return GDN_ERR_SHAPE;
  if ((int64_t)c->max_pages * c->page_size > kMaxPositions) return GDN_ERR_SHAPE;
  // a pool's rows are counted in 64 bits; its bytes must fit a size_t with room to spare
  if ((double)c->num_pages * c->num_kv_heads * c->page_size * c->head_dim > 4e15) return GDN_ERR_SHAPE;
  if (!pointers) return GDN_OK;
  const bool e4m3 = c->format == GDN_CACHE_E4M3;
  if (c->k_pages == nullptr || c->v_pages == nullptr || c->page_table == nullptr) return GDN_ERR_NULL;
  if (e4m3 && (c->k_scales == nullptr || c->v_scales == nullptr)) return GDN_ERR_NULL;
  if (!e4m3 && (c->k_scales != nullptr || c->v_scales != nullptr)) return GDN_ERR_SHAPE;
  for (const void* ptr : {c->k_pages, c->v_pages, (void*)c->k_scales, (void*)c->v_scales})
    if (ptr != nullptr && !aligned16(ptr)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

struct CacheSpans {
  Span pages[2], scales[2], table;
  CacheSpans(const gdn_kv_cache& c, int64_t R) {
    const bool e4m3 = c.format == GDN_CACHE_E4M3;
    const size_t rows = (size_t)c.num_pages * c.num_kv_heads * c.page_size;
    const size_t bytes = rows * c.head_dim * (e4m3 ? 1 : io_bytes(c.io_dtype));
    pages[0] = Span(c.k_pages, bytes);
    pages[1] = Span(c.v_pages, bytes);
    scales[0] = Span(c.k_scales, e4m3 ? rows : 0);
    scales[1] = Span(c.v_scales, e4m3 ? rows : 0);
    table = Span(c.page_table, (size_t)R * c.max_pages * 4);
  }
  bool overlap_each_other() const {
    const Span* all[] = {&pages[0], &pages[1], &scales[0], &scales[1], &table};
    for (int i = 0; i < 5; ++i)
      for (int j = i + 1; j < 5; ++j)
        if (all[i]->overlaps(*all[j])) return true;
    return false;
  }
  template <typename S> bool overlap_pool(const S& s) const {
    return s.overlaps(pages[0]) || s.overlaps(pages[1]) || s.overlaps(scales[0]) || s.overlaps(scales[1]);
  }
  template <typename S> bool overlap(const S& s) const { return overlap_pool(s) || s.overlaps(table); }
};

// The packing of the call and the cached lengths, and what their host mirrors say.
struct Rows {
  int64_t N, R;
  const int32_t *cu, *cu_host, *lens, *lens_host;
  bool dense() const { return cu == nullptr; }
  int64_t dense_len() const { return R > 0 ? N / R : 0; }
  // T_r where the host knows it, else -1
  int64_t tokens(int64_t r) const {
    return dense() ? dense_len() : cu_host != nullptr ? (int64_t)cu_host[r + 1] - cu_host[r] : -1;
  }
};

int check_rows(const Rows& w, const gdn_kv_cache& c) {
  if (w.dense() && (w.cu_host != nullptr || w.N % w.R != 0)) return GDN_ERR_SHAPE;
  if (w.lens == nullptr) return GDN_ERR_NULL;
  if (w.cu_host != nullptr && !gdn::cu_host_ok(w.cu_host, w.R, w.N)) return GDN_ERR_SHAPE;
  if (w.lens_host != nullptr)
    for (int64_t r = 0; r < w.R; ++r)
      if (w.lens_host[r] < std::max<int64_t>(w.tokens(r), 0) ||
          w.lens_host[r] > (int64_t)c.max_pages * c.page_size)
        return GDN_ERR_CAPACITY;
  if (c.page_table_host != nullptr)
    for (int64_t i = 0; i < w.R * c.max_pages; ++i)
      if (c.page_table_host[i] < -1 || c.page_table_host[i] >= c.num_pages) return GDN_ERR_SHAPE;
  return GDN_OK;
}

// Whether two requests write one page, as far as the host mirrors show. (A page
// twice in one request's table is not looked for.)
bool pages_collide(const Rows& w, const gdn_kv_cache& c) {
  if (c.page_table_host == nullptr || w.lens_host == nullptr || (!w.dense() && w.cu_host == nullptr)) return false;
  auto first = [&](int64_t r) { return (w.lens_host[r] - w.tokens(r)) / c.page_size; };
  auto past = [&](int64_t r) { return w.tokens(r) > 0 ? (w.lens_host[r] - 1) / c.page_size + 1 : first(r); };
  size_t n = 0;
  for (int64_t r = 0; r < w.R; ++r) n += (size_t)(past(r) - first(r));
  typedef std::pair<int32_t, int32_t> Use;       // (page, request)
  Use* uses = new (std::nothrow) Use[n + 1];
  if (uses == nullptr) return false;
  size_t m = 0;
  for (int64_t r = 0; r < w.R; ++r)
    for (int64_t i = first(r); i < past(r); ++i) {
      const int32_t page = c.page_table_host[r * c.max_pages + i];
      if (page >= 0) uses[m++] = Use(page, (int32_t)r);
    }
  std::sort(uses, uses + m);
  bool twice = false;
  for (size_t i = 1; i < m; ++i)
    twice = twice || (uses[i].first == uses[i - 1].first && uses[i].second != uses[i - 1].second);
  delete[] uses;
  return twice;
}

gdn::CacheArgs cache_args(const gdn_kv_cache& c) {
  gdn::CacheArgs a{};
  a.k = c.k_pages; a.v = c.v_pages; a.k_scales = c.k_scales; a.v_scales = c.v_scales; a.table = c.page_table;
  a.num_pages = c.num_pages; a.max_pages = c.max_pages; a.Hk = c.num_kv_heads; a.D = c.head_dim;
  a.e4m3 = c.format == GDN_CACHE_E4M3 ? 1 : 0;
  while ((1 << a.page_shift) < c.page_size) ++a.page_shift;
  return a;
}

gdn::RowArgs row_args(const Rows& w) {
  gdn::RowArgs a{};
  a.cu_seqlens = w.cu; a.seq_lens = w.lens;
  a.N = (int32_t)w.N; a.R = (int32_t)w.R; a.dense_len = w.dense() ? (int32_t)w.dense_len() : 0;
  return a;
}

// Tokens per workgroup of the rotation and cache kernels: about two items (32 bytes of
// a head each) a thread, and at least 4 workgroups per CU where there are tokens for
// them. More tokens leave fewer workgroups with more items in a row, and too little
// in flight: 15,352 tokens of 28 heads x 256 fp16, one a workgroup 76 us, 4 90 us,
// 14 99 us; reading 32,768 tokens of 4 key heads, 1, 2, 4, 8 a workgroup 45, 34, 31,
// 39 us.
int tokens_per_block(int64_t N, int64_t heads, int64_t D, size_t io) {
  const int64_t items = heads * D * (int64_t)io / 32;
  const int64_t t = std::min<int64_t>(512 / std::max<int64_t>(items, 1), N / 1024);
  return (int)std::min<int64_t>(std::max<int64_t>(t, 1), gdn::kRopeMaxTokens);
}

int status_of(hipError_t err) { return err == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

}  // namespace

extern "C" {

int gdn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double scale, double trained_length,
                         double beta_fast, double beta_slow, double* inv_freq, float* factor) {
  if (inv_freq == nullptr || factor == nullptr) return GDN_ERR_NULL;
  if (scaling < GDN_ROPE_SCALING_NONE || scaling > GDN_ROPE_SCALING_YARN) return GDN_ERR_RULE;
  const int r = rotary_dim;
  if (r < 2 || r % 2 != 0 || !std::isfinite(base) || !(base > 1.0)) return GDN_ERR_SHAPE;
  if (scaling != GDN_ROPE_SCALING_NONE && (!std::isfinite(scale) || !(scale > 0.0))) return GDN_ERR_SHAPE;
  double lo = 0, hi = 0;
  if (scaling == GDN_ROPE_SCALING_NTK) {
    if (r < 4) return GDN_ERR_SHAPE;
    base *= std::pow(scale, r / (r - 2.0));
    if (!std::isfinite(base) || !(base > 0.0)) return GDN_ERR_SHAPE;
  } else if (scaling == GDN_ROPE_SCALING_YARN) {
    if (!std::isfinite(trained_length) || !(trained_length > 0.0) || !std::isfinite(beta_fast) ||
        !std::isfinite(beta_slow))
      return GDN_ERR_SHAPE;
    const double fast = beta_fast > 0.0 ? beta_fast : 32.0, slow = beta_slow > 0.0 ? beta_slow : 1.0;
    auto at = [&](double turns) { return r * std::log(trained_length / (turns * 2.0 * kPi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(at(fast)), 0.0);
    hi = std::min(std::ceil(at(slow)), r - 1.0);
  }
  for (int i = 0; i < r / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    inv_freq[i] = f;
    if (scaling == GDN_ROPE_SCALING_LINEAR) inv_freq[i] = f / scale;
    if (scaling == GDN_ROPE_SCALING_YARN) {
      const double w = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      inv_freq[i] = f * (1.0 - w) + f / scale * w;
    }
  }
  *factor = scaling == GDN_ROPE_SCALING_YARN && scale > 1.0 ? (float)(0.1 * std::log(scale) + 1.0) : 1.0f;
  return GDN_OK;
}

int gdn_rope_forward(const gdn_rope_params* p, const gdn_rope_tensors* t, void* stream) {
  if (p == nullptr || t == nullptr) return GDN_ERR_NULL;
  if (p->layout != GDN_ROPE_HALF && p->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_RULE;
  if (!std::isfinite(p->factor)) return GDN_ERR_RULE;
  if (p->io_dtype != GDN_F32 && p->io_dtype != GDN_F16) return GDN_ERR_DTYPE;
  const int64_t N = p->num_tokens, Hq = p->num_q_heads, Hk = p->num_k_heads, D = p->head_dim;
  if (N < 0 || Hq < 0 || Hk < 0 || !head_dim_ok(p->head_dim)) return GDN_ERR_SHAPE;
  if ((Hq + Hk) * D > std::numeric_limits<int32_t>::max()) return GDN_ERR_SHAPE;
  if (p->rotary_dim < 16 || p->rotary_dim > D || p->rotary_dim % 16 != 0) return GDN_ERR_SHAPE;
  const int64_t qs = token_stride(p->q_stride, Hq, D), ks = token_stride(p->k_stride, Hk, D);
  if (qs < 0 || ks < 0) return GDN_ERR_SHAPE;
  if (N == 0 || Hq + Hk == 0) return GDN_OK;
  if ((Hq > 0 && (t->q == nullptr || t->q_out == nullptr)) || (Hk > 0 && (t->k == nullptr || t->k_out == nullptr)) ||
      t->positions == nullptr || t->inv_freq == nullptr)
    return GDN_ERR_NULL;
  for (const void* ptr : {t->q, t->k, (const void*)t->q_out, (const void*)t->k_out, (const void*)t->inv_freq})
    if (ptr != nullptr && !aligned16(ptr)) return GDN_ERR_SHAPE;
  const size_t io = io_bytes(p->io_dtype);
  const bool q_in = t->q_out == t->q, k_in = t->k_out == t->k;
  const int64_t qos = q_in ? qs : Hq * D, kos = k_in ? ks : Hk * D;
  const RowSpan q(t->q, Hq * D * io, qs * io, N), k(t->k, Hk * D * io, ks * io, N);
  const RowSpan qo(t->q_out, Hq * D * io, qos * io, N), ko(t->k_out, Hk * D * io, kos * io, N);
  const Span pos(t->positions, N * 4), freq(t->inv_freq, (size_t)p->rotary_dim / 2 * 8);
  if ((!q_in && qo.overlaps(q)) || (!k_in && ko.overlaps(k)) || qo.overlaps(k) || ko.overlaps(q) || qo.overlaps(ko))
    return GDN_ERR_ALIAS;
  for (const Span& s : {pos, freq})
    if (qo.overlaps(s) || ko.overlaps(s)) return GDN_ERR_ALIAS;

  gdn::RopeArgs a{};
  a.q = t->q; a.k = t->k; a.q_out = t->q_out; a.k_out = t->k_out;
  a.positions = t->positions; a.inv_freq = t->inv_freq;
  a.N = (int32_t)N; a.Hq = (int32_t)Hq; a.Hk = (int32_t)Hk; a.D = (int32_t)D;
  a.rot = p->rotary_dim; a.interleaved = p->layout == GDN_ROPE_INTERLEAVED ? 1 : 0;
  a.factor = p->factor == 0.f ? 1.f : p->factor;
  a.q_stride = qs; a.k_stride = ks; a.q_out_stride = qos; a.k_out_stride = kos;
  a.q_in_place = q_in ? 1 : 0; a.k_in_place = k_in ? 1 : 0;
  a.tokens_per_block = tokens_per_block(N, Hq + Hk, D, io);
  return status_of(gdn::launch_rope(a, p->io_dtype, static_cast<hipStream_t>(stream)));
}

int gdn_kv_write(const gdn_kv_params* p, const gdn_kv_tensors* t, const gdn_kv_cache* c, void* stream) {
  if (p == nullptr || t == nullptr) return GDN_ERR_NULL;
  int st = check_cache(c, false);
  if (st != GDN_OK) return st;
  const int64_t N = p->num_tokens, R = p->num_reqs, Hq = p->num_q_heads, Hk = c->num_kv_heads, D = c->head_dim;
  if (N < 0 || R < 0 || Hq < 0) return GDN_ERR_SHAPE;
  if ((Hq + 2 * Hk) * D > std::numeric_limits<int32_t>::max()) return GDN_ERR_SHAPE;
  const bool rotate = p->rotary_dim != 0;
  if (rotate && (p->rotary_dim < 16 || p->rotary_dim > D || p->rotary_dim % 16 != 0)) return GDN_ERR_SHAPE;
  if (!rotate && Hq != 0) return GDN_ERR_SHAPE;
  if (rotate && p->rope_layout != GDN_ROPE_HALF && p->rope_layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_RULE;
  if (rotate && !std::isfinite(p->rope_factor)) return GDN_ERR_RULE;
  const int64_t qs = token_stride(p->q_stride, Hq, D), ks = token_stride(p->k_stride, Hk, D),
                vs = token_stride(p->v_stride, Hk, D);
  if (qs < 0 || ks < 0 || vs < 0) return GDN_ERR_SHAPE;
  if (R == 0) return N == 0 ? GDN_OK : GDN_ERR_SHAPE;
  st = check_cache(c, true);
  if (st != GDN_OK) return st;
  const Rows w{N, R, t->cu_seqlens, t->cu_seqlens_host, t->seq_lens, t->seq_lens_host};
  st = check_rows(w, *c);
  if (st != GDN_OK) return st;
  if (N == 0) return GDN_OK;
  if (t->k == nullptr || t->v == nullptr) return GDN_ERR_NULL;
  if (rotate && t->inv_freq == nullptr) return GDN_ERR_NULL;
  if (Hq > 0 && (t->q == nullptr || t->q_out == nullptr)) return GDN_ERR_NULL;
  for (const void* ptr : {(const void*)t->k, (const void*)t->v, t->q, (const void*)t->q_out, (const void*)t->inv_freq})
    if (ptr != nullptr && !aligned16(ptr)) return GDN_ERR_SHAPE;
  const size_t io = io_bytes(c->io_dtype);
  const bool q_in = t->q_out == t->q;
  const int64_t qos = q_in ? qs : Hq * D;
  const RowSpan q(t->q, Hq * D * io, qs * io, N), qo(t->q_out, Hq * D * io, qos * io, N);
  const RowSpan k(t->k, Hk * D * io, ks * io, N), v(t->v, Hk * D * io, vs * io, N);
  const CacheSpans cs(*c, R);
  if (cs.overlap_each_other()) return GDN_ERR_ALIAS;
  const Span ints[] = {Span(t->cu_seqlens, (R + 1) * 4), Span(t->seq_lens, R * 4),
                       Span(rotate ? t->positions : nullptr, N * 4),
                       Span(rotate ? t->inv_freq : nullptr, (size_t)p->rotary_dim / 2 * 8)};
  for (const Span& s : ints)
    if (cs.overlap_pool(s) || (Hq > 0 && qo.overlaps(s))) return GDN_ERR_ALIAS;
  if (cs.overlap_pool(k) || cs.overlap_pool(v)) return GDN_ERR_ALIAS;
  if (Hq > 0 && (cs.overlap_pool(q) || cs.overlap(qo) || (!q_in && qo.overlaps(q)) || qo.overlaps(k) || qo.overlaps(v)))
    return GDN_ERR_ALIAS;
  if (pages_collide(w, *c)) return GDN_ERR_ALIAS;

  gdn::RopeArgs a{};
  a.q = t->q; a.k = t->k; a.v = t->v; a.q_out = t->q_out;
  a.positions = t->positions; a.inv_freq = t->inv_freq;
  a.N = (int32_t)N; a.Hq = (int32_t)Hq; a.Hk = (int32_t)Hk; a.D = (int32_t)D;
  a.rot = p->rotary_dim; a.interleaved = p->rope_layout == GDN_ROPE_INTERLEAVED ? 1 : 0;
  a.factor = p->rope_factor == 0.f ? 1.f : p->rope_factor;
  a.q_stride = qs; a.k_stride = ks; a.v_stride = vs; a.q_out_stride = qos;
  a.q_in_place = q_in ? 1 : 0;
  a.tokens_per_block = tokens_per_block(N, Hq + 2 * Hk, D, io);
  a.to_cache = 1;
  a.cache = cache_args(*c);
  a.rows = row_args(w);
  return status_of(gdn::launch_rope(a, c->io_dtype, static_cast<hipStream_t>(stream)));
}

int gdn_kv_read(const gdn_kv_params* p, const gdn_kv_tensors* t, const gdn_kv_cache* c, void* stream) {
  if (p == nullptr || t == nullptr) return GDN_ERR_NULL;
  int st = check_cache(c, false);
  if (st != GDN_OK) return st;
  const int64_t N = p->num_tokens, R = p->num_reqs, Hk = c->num_kv_heads, D = c->head_dim;
  if (N < 0 || R < 0 || p->num_q_heads != 0 || p->rotary_dim != 0) return GDN_ERR_SHAPE;
  if (p->q_stride != 0 || p->k_stride != 0 || p->v_stride != 0) return GDN_ERR_SHAPE;     // dense rows only
  if (2 * Hk * D > std::numeric_limits<int32_t>::max()) return GDN_ERR_SHAPE;
  if (R == 0) return N == 0 ? GDN_OK : GDN_ERR_SHAPE;
  st = check_cache(c, true);
  if (st != GDN_OK) return st;
  const Rows w{N, R, t->cu_seqlens, t->cu_seqlens_host, t->seq_lens, t->seq_lens_host};
  st = check_rows(w, *c);
  if (st != GDN_OK) return st;
  if (N == 0) return GDN_OK;
  if (t->k == nullptr || t->v == nullptr) return GDN_ERR_NULL;
  if (!aligned16(t->k) || !aligned16(t->v)) return GDN_ERR_SHAPE;
  const size_t bytes = (size_t)N * Hk * D * io_bytes(c->io_dtype);
  const Span k(t->k, bytes), v(t->v, bytes), cu(t->cu_seqlens, (R + 1) * 4), lens(t->seq_lens, R * 4);
  const CacheSpans cs(*c, R);
  if (k.overlaps(v) || cs.overlap(k) || cs.overlap(v)) return GDN_ERR_ALIAS;
  for (const Span& s : {cu, lens})
    if (k.overlaps(s) || v.overlaps(s)) return GDN_ERR_ALIAS;
  gdn::ReadArgs a{};
  a.k = t->k; a.v = t->v;
  a.tokens_per_block = tokens_per_block(N, 2 * Hk, D, io_bytes(c->io_dtype));
  a.cache = cache_args(*c);
  a.rows = row_args(w);
  return status_of(gdn::launch_kv_read(a, c->io_dtype, static_cast<hipStream_t>(stream)));
}

static int check_attn(const gdn_attn_params* p, const gdn_kv_cache* c, int64_t* q_stride) {
  if (p == nullptr) return GDN_ERR_NULL;
  const int st = check_cache(c, false);
  if (st != GDN_OK) return st;
  const int64_t N = p->num_tokens, R = p->num_reqs, Hq = p->num_q_heads, D = c->head_dim;
  if (N < 0 || R < 0 || Hq < 1 || Hq % c->num_kv_heads != 0 || p->window < 0) return GDN_ERR_SHAPE;
  if (Hq * D > std::numeric_limits<int32_t>::max()) return GDN_ERR_SHAPE;
  if (std::isnan(p->scale) || std::isinf(p->scale)) return GDN_ERR_SHAPE;
  // workgroups are numbered by (token, query head, 64 columns), and units of work counted, in 32 bits
  if ((N + R) * Hq * (D / 64) > ((int64_t)1 << 30)) return GDN_ERR_SHAPE;
  *q_stride = token_stride(p->q_stride, Hq, D);
  return *q_stride < 0 ? GDN_ERR_SHAPE : GDN_OK;
}

int gdn_attn_workspace_bytes(const gdn_attn_params* p, const gdn_kv_cache* c, size_t* bytes) {
  int64_t qs = 0;
  const int st = check_attn(p, c, &qs);
  if (st != GDN_OK) return st;
  if (bytes == nullptr) return GDN_ERR_NULL;
  *bytes = gdn::attn_workspace_bytes(p->num_tokens, p->num_reqs, p->num_q_heads, c->num_kv_heads, c->head_dim);
  return GDN_OK;
}

int gdn_attn_forward(const gdn_attn_params* p, const gdn_attn_tensors* t, const gdn_kv_cache* c, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int64_t qs = 0;
  int st = check_attn(p, c, &qs);
  if (st != GDN_OK) return st;
  if (t == nullptr) return GDN_ERR_NULL;
  const int64_t N = p->num_tokens, R = p->num_reqs, Hq = p->num_q_heads, Hk = c->num_kv_heads, D = c->head_dim;
  if (R == 0) return N == 0 ? GDN_OK : GDN_ERR_SHAPE;
  st = check_cache(c, true);
  if (st != GDN_OK) return st;
  const Rows w{N, R, t->cu_seqlens, t->cu_seqlens_host, t->seq_lens, t->seq_lens_host};
  st = check_rows(w, *c);
  if (st != GDN_OK) return st;
  if (N == 0) return GDN_OK;
  if (t->q == nullptr || t->output == nullptr) return GDN_ERR_NULL;
  if (!aligned16(t->q) || !aligned16(t->output)) return GDN_ERR_SHAPE;
  const size_t need = gdn::attn_workspace_bytes(N, R, (int)Hq, (int)Hk, (int)D);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))) return GDN_ERR_WORKSPACE;
  const size_t io = io_bytes(c->io_dtype);
  const RowSpan q(t->q, Hq * D * io, qs * io, N);
  const Span out(t->output, (size_t)N * Hq * D * io), ws(workspace, need);
  const Span cu(t->cu_seqlens, (R + 1) * 4), lens(t->seq_lens, R * 4);
  const CacheSpans cs(*c, R);
  for (const Span& o : {out, ws})
    if (q.overlaps(o) || cs.overlap(o) || o.overlaps(cu) || o.overlaps(lens)) return GDN_ERR_ALIAS;
  if (out.overlaps(ws)) return GDN_ERR_ALIAS;
  gdn::AttnArgs a{};
  a.q = t->q; a.output = t->output; a.q_stride = qs;
  a.Hq = (int32_t)Hq; a.group = (int32_t)(Hq / Hk); a.window = p->window;
  a.scale = p->scale > 0.f ? p->scale : 1.0f / std::sqrt((float)D);
  // the most tokens of a request, and the most positions one attends, as far as they are known here: a
  // mirror's, else what the call and the table hold
  int64_t tokens = N, longest = (int64_t)c->max_pages * c->page_size;
  if (w.dense()) tokens = w.dense_len();
  if (w.cu_host != nullptr) {
    tokens = 0;
    for (int64_t r = 0; r < R; ++r) tokens = std::max(tokens, w.tokens(r));
  }
  int64_t sum = 0;
  if (p->window > 0) longest = std::min(longest, (int64_t)p->window + tokens);
  if (w.lens_host != nullptr) {
    const int64_t most = longest;
    longest = 0;
    for (int64_t r = 0; r < R; ++r) {
      const int64_t n = std::min<int64_t>(w.lens_host[r], most);
      longest = std::max(longest, n);
      sum += n;
    }
  }
  a.max_tokens = (int32_t)tokens;
  a.max_len = (int32_t)longest;
  a.sum_len = sum;
  a.cache = cache_args(*c);
  a.rows = row_args(w);
  return status_of(gdn::launch_attn(a, c->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

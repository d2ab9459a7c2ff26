// Internal launch interface between the C ABI (gdn_attn_api.cpp) and the HIP
// kernels of the attention layer: rotary positions, paged cache, attention.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// The paged cache of one layer (gdn_kv_cache); pages [P, Hk, page_size, D].
struct CacheArgs {
  void* k;
  void* v;
  uint8_t* k_scales;            // null unless e4m3
  uint8_t* v_scales;
  const int32_t* table;         // [R, max_pages]
  int32_t num_pages, page_shift, max_pages, Hk, D;
  int32_t e4m3;
};

// The packed tokens of a call and the cached tokens of their requests.
struct RowArgs {
  const int32_t* cu_seqlens;    // null: dense layout, dense_len tokens per request
  const int32_t* seq_lens;      // [R]
  int32_t N, R, dense_len;
};

// First token of request i (i = R: the end of the last), clamped to [0, N].
__host__ __device__ inline int row_start(const RowArgs& p, int i) {
  const int64_t x = p.cu_seqlens != nullptr ? (int64_t)p.cu_seqlens[i] : (int64_t)i * p.dense_len;
  return (int)(x < 0 ? 0 : x > p.N ? p.N : x);
}

// Row (page * Hk + head 0) * page_size + slot of a request's position in the
// pool, or -1 where no page holds it. Head h's row is h * page_size further.
__device__ inline int64_t cache_row(const CacheArgs& c, int r, int64_t pos) {
  if (pos < 0 || pos >= ((int64_t)c.max_pages << c.page_shift)) return -1;
  const int page = c.table[(int64_t)r * c.max_pages + (pos >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) return -1;
  return (((int64_t)page * c.Hk) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Rotation of q and k, and the write of k and v to the cache.
struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;                // cache write only
  void* q_out;
  void* k_out;                  // null with the cache write
  const int32_t* positions;     // null: the positions in the cache
  const double* inv_freq;
  int32_t N, Hq, Hk, D;
  int32_t rot;                  // rotary_dim; 0: no rotation
  int32_t interleaved;
  float factor;
  int64_t q_stride, k_stride, v_stride;      // elements between tokens of the inputs
  int64_t q_out_stride, k_out_stride;
  int32_t q_in_place, k_in_place;
  int32_t tokens_per_block;
  int32_t to_cache;
  CacheArgs cache;
  RowArgs rows;
};

struct ReadArgs {
  void* k;
  void* v;
  int32_t tokens_per_block;
  CacheArgs cache;
  RowArgs rows;
};

struct AttnArgs {
  const void* q;
  void* output;
  int64_t q_stride;
  int32_t Hq, group;            // group = Hq / Hk
  int32_t window;               // 0: none
  int32_t max_len;              // no request attends more positions, as far as the host knows
  int64_t sum_len;              // attended positions of all requests, 0 where the host does not know
  int32_t max_tokens;           // no request has more tokens, as far as the host knows
  float scale;
  CacheArgs cache;
  RowArgs rows;
};

constexpr int kRopeMaxTokens = 16;   // tokens one workgroup of the rotation and cache kernels handles

// io_dtype: 0 = f32, 1 = f16 (gdn_dtype values).
hipError_t launch_rope(const RopeArgs& args, int io_dtype, hipStream_t stream);
hipError_t launch_kv_read(const ReadArgs& args, int io_dtype, hipStream_t stream);
hipError_t launch_attn(const AttnArgs& args, int io_dtype, void* workspace, hipStream_t stream);

// Workspace bytes of the attention for N tokens of R requests.
size_t attn_workspace_bytes(int64_t N, int64_t R, int Hq, int Hk, int D);

}  // namespace gdn

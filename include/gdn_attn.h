/*
 * gdn_attn.h - C ABI of the full-attention layers' serving step in libgdn.so.
 *
 * A hybrid model interleaves its GatedDeltaNet layers with full-attention
 * layers, whose per-request state is not one fixed block but a cache of keys
 * and values in pages ("Replay compact fixed state for hybrid decoding", Key
 * Changes: paged and fixed state groups side by side; "Add GatedDeltaNet
 * evaluation export for Qwen hybrid models", What changed). The entry points
 * here are those layers' counterparts of gdn_forward on the same packed or
 * dense tokens (one token per request, a few draft tokens, or prompts):
 *
 *   gdn_rope_forward   rotary positions on q and k
 *   gdn_kv_write       the new tokens' keys and values into the pages, with the
 *                      rotation of q and k fused on request
 *   gdn_kv_read        cached tokens back as packed keys and values
 *   gdn_attn_forward   attention of every request's newest tokens over its pages
 *
 * Draft tokens that are not accepted need no replay: the caller leaves
 * seq_lens behind them and the next step overwrites them.
 *
 * Conventions as in gdn.h: the caller owns every buffer, the library allocates
 * no device memory and keeps no pointer, every check runs on the host before
 * anything is enqueued (a status other than GDN_ERR_HIP means no device write),
 * all work is asynchronous on `stream` and can be captured in a HIP graph, and
 * the status codes are gdn_status. "io" is the element type named by io_dtype,
 * GDN_F16 or GDN_F32 (BF16 is rejected). Device pointers are 16-byte aligned
 * unless they are int32 arrays.
 */
#ifndef GDN_ATTN_H_
#define GDN_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- The paged cache.
 *
 * A pool of num_pages pages holds page_size tokens' keys (or values) each, head
 * by head, so that one head's tokens of a page are contiguous:
 *   k_pages, v_pages  [num_pages, num_kv_heads, page_size, head_dim]
 * page_table[r][i] is the page of request r's positions i * page_size ..
 * (i + 1) * page_size - 1.
 *
 * Formats:
 *  GDN_CACHE_IO    the pages hold io elements.
 *  GDN_CACHE_E4M3  (GDN_F16 io only) the pages hold 8-bit floats (e4m3: 4 exponent
 *                  bits, 3 mantissa bits, largest value 448), and k_scales, v_scales
 *                  [num_pages, num_kv_heads, page_size] an exponent byte s per row of
 *                  head_dim elements: element = code * 2^(s - 127). Writing takes
 *                  a = the largest finite |x| of the row, 2^(s - 127) = the smallest
 *                  power of two with a <= 448 * 2^(s - 127), and code = x / 2^(s - 127)
 *                  rounded to nearest even; s = 0 when no finite x is nonzero, and a
 *                  non-finite x is stored as NaN. A power of two makes the division and
 *                  the way back exact, so a code is the only rounding. Rows of FP16 have
 *                  s = 0 or 95 .. 135, and no other byte may stand beside a position that
 *                  is attended (attention takes a value's byte below 94 as 94).
 *
 * A page number outside [0, num_pages) (e.g. -1) names no page: nothing is
 * written there, reads give zeros, and attention leaves those positions out.
 * The same holds for positions outside [0, max_pages * page_size). */
typedef enum gdn_cache_format { GDN_CACHE_IO = 0, GDN_CACHE_E4M3 = 1 } gdn_cache_format;

typedef struct gdn_kv_cache {
  void* k_pages;
  void* v_pages;
  uint8_t* k_scales;              /* GDN_CACHE_E4M3 only, else NULL                  */
  uint8_t* v_scales;
  const int32_t* page_table;      /* device, i32 [R, max_pages]                      */
  const int32_t* page_table_host; /* host mirror or NULL. When given every entry must
                                     lie in [-1, num_pages), else GDN_ERR_SHAPE      */
  int32_t num_pages;              /* >= 1                                            */
  int32_t page_size;              /* 16, 32, 64, 128, 256, 512 or 1024 tokens         */
  int32_t max_pages;              /* >= 1; max_pages * page_size <= 2^30              */
  int32_t num_kv_heads;           /* Hk >= 1                                         */
  int32_t head_dim;               /* D in {64, 128, 256}                             */
  int32_t io_dtype;               /* gdn_dtype of q, k, v and outputs                */
  int32_t format;                 /* gdn_cache_format                                */
} gdn_kv_cache;

/* ---- Rotary positions.
 *
 * With the angle t = position * inv_freq[i] of pair i, c = factor cos t and
 * s = factor sin t, the pair (x, y) becomes (x c - y s, y c + x s). The pairs of
 * the leading rotary_dim = r elements of a head are
 *   GDN_ROPE_HALF         (i, i + r / 2)
 *   GDN_ROPE_INTERLEAVED  (2 i, 2 i + 1)           i = 0 .. r / 2 - 1
 * and the elements from r on are left as they are. Frequencies are doubles; the angle is
 * formed and reduced without rounding it, so that far positions lose nothing, and its
 * cos and sin times the factor are rounded once to FP32. The rotation itself
 * runs in FP32 and is rounded once to io. */
typedef enum gdn_rope_layout { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;

/* Frequencies for contexts longer than the trained one, with f_i = base^(-2 i / r)
 * and s = scale:
 *  GDN_ROPE_SCALING_NONE    f_i
 *  GDN_ROPE_SCALING_LINEAR  f_i / s                       (position interpolation)
 *  GDN_ROPE_SCALING_NTK     (base s^(r / (r - 2)))^(-2 i / r)
 *  GDN_ROPE_SCALING_YARN    f_i (1 - w_i) + f_i / s w_i, w_i a ramp from 0 to 1 over the
 *                           pair indices lo .. hi; with d(n) = r ln(trained_length / (2 pi n))
 *                           / (2 ln base), the index that turns n times within the trained
 *                           length, lo = max(floor(d(beta_fast)), 0), hi = min(ceil(d(beta_slow)),
 *                           r - 1), w_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1); the factor
 *                           is 0.1 ln s + 1 (1 for s <= 1). */
typedef enum gdn_rope_scaling {
  GDN_ROPE_SCALING_NONE = 0,
  GDN_ROPE_SCALING_LINEAR = 1,
  GDN_ROPE_SCALING_NTK = 2,
  GDN_ROPE_SCALING_YARN = 3
} gdn_rope_scaling;

/* Writes the rotary_dim / 2 frequencies to inv_freq (HOST memory) and the
 * multiplier of cos and sin to *factor. A host computation: nothing is enqueued.
 * trained_length, beta_fast and beta_slow are read by YARN only (<= 0 selects 32
 * and 1 for the betas). Errors: GDN_ERR_NULL; GDN_ERR_RULE for an unknown scaling;
 * GDN_ERR_SHAPE for rotary_dim not a positive even number (NTK: at least 4), base
 * <= 1, scale <= 0, a non-finite argument, or YARN without a trained length. */
int gdn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double scale, double trained_length,
                         double beta_fast, double beta_slow, double* inv_freq, float* factor);

typedef struct gdn_rope_params {
  int32_t num_tokens;            /* N >= 0                                          */
  int32_t num_q_heads;           /* Hq >= 0                                         */
  int32_t num_k_heads;           /* Hk >= 0                                         */
  int32_t head_dim;              /* D in {64, 128, 256}                             */
  int32_t io_dtype;              /* GDN_F16 or GDN_F32                              */
  int32_t rotary_dim;            /* r: a multiple of 16, 16 .. D                    */
  int32_t layout;                /* gdn_rope_layout                                 */
  float factor;                  /* of cos and sin; 0 selects 1                     */
  int32_t q_stride;              /* elements from one token's q to the next's; 0:
                                    Hq * D. At least Hq * D, a multiple of 8        */
  int32_t k_stride;              /* likewise of k                                   */
} gdn_rope_params;

typedef struct gdn_rope_tensors {
  const void* q;                 /* device, io [N, Hq, D], rows q_stride apart       */
  const void* k;                 /* device, io [N, Hk, D], rows k_stride apart       */
  const int32_t* positions;      /* device, i32 [N]; any value                      */
  const double* inv_freq;        /* device, f64 [r / 2]                             */
  void* q_out;                   /* device, io [N, Hq, D] dense, or q itself: then in
                                    place, with q's stride, and the elements from r on
                                    are neither read nor written                     */
  void* k_out;                   /* likewise for k                                  */
} gdn_rope_tensors;

/* Rotates q and k. q (k) and its output may be NULL when Hq (Hk) is 0. Errors:
 * GDN_ERR_NULL, GDN_ERR_SHAPE (sizes, strides or alignment), GDN_ERR_DTYPE,
 * GDN_ERR_RULE (unknown layout, non-finite factor), GDN_ERR_ALIAS (an output overlaps an input other
 * than in place, or the other output). */
int gdn_rope_forward(const gdn_rope_params* params, const gdn_rope_tensors* tensors, void* stream);

/* ---- Writing and reading the cache.
 *
 * The tokens of a call are packed as in gdn.h: request r owns tokens cu_seqlens[r]
 * .. cu_seqlens[r + 1] - 1, T_r of them (cu_seqlens NULL: N / R each). They are the
 * newest T_r of the seq_lens[r] tokens that the request has in the cache once this
 * call is done: token j has position seq_lens[r] - T_r + j. */
typedef struct gdn_kv_params {
  int32_t num_tokens;            /* N >= 0                                          */
  int32_t num_reqs;              /* R >= 0                                          */
  int32_t num_q_heads;           /* gdn_kv_write with a rotation: Hq >= 0; else 0    */
  int32_t rotary_dim;            /* gdn_kv_write: 0 for no rotation, else as in
                                    gdn_rope_params; gdn_kv_read: 0                  */
  int32_t rope_layout;           /* gdn_rope_layout                                 */
  float rope_factor;             /* 0 selects 1                                     */
  int32_t q_stride;              /* as in gdn_rope_params                           */
  int32_t k_stride;
  int32_t v_stride;
} gdn_kv_params;

typedef struct gdn_kv_tensors {
  void* k;                       /* device, io [N, Hk, D]: gdn_kv_write reads rows
                                    k_stride apart; gdn_kv_read writes dense rows    */
  void* v;                       /* likewise                                        */
  const int32_t* cu_seqlens;     /* device, i32 [R + 1], or NULL                    */
  const int32_t* cu_seqlens_host;/* host mirror or NULL, as in gdn.h: what it says
                                    must be what cu_seqlens holds when the work runs,
                                    so a captured call whose cu_seqlens changes
                                    between replays gives none                      */
  const int32_t* seq_lens;       /* device, i32 [R]                                 */
  const int32_t* seq_lens_host;  /* host mirror or NULL; every value must lie in
                                    [T_r, max_pages * page_size], else
                                    GDN_ERR_CAPACITY (T_r is checked where the host
                                    knows it). Besides the checks it only guides how
                                    the work is split: a captured call may be replayed
                                    with other lengths. The split stays the captured
                                    one, so gdn_attn_forward captured with short
                                    lengths is slow over far longer ones (one request,
                                    300 positions at capture and 131,072 at replay, 8
                                    key heads of 128 FP16: 1.4 ms instead of 92 us):
                                    capture it with the longest to come, or with NULL,
                                    which counts as the table's length               */
  const void* q;                 /* with rotary_dim > 0 and Hq > 0: rotated into q_out */
  void* q_out;                   /* io [N, Hq, D] dense, or q itself (in place)      */
  const int32_t* positions;      /* device, i32 [N]: rotary positions, or NULL for
                                    the positions in the cache                      */
  const double* inv_freq;        /* device, f64 [rotary_dim / 2]                    */
} gdn_kv_tensors;

/* Writes the tokens' keys and values to their pages; with rotary_dim > 0 the keys are
 * rotated first, and q into q_out: the same bytes as gdn_rope_forward followed by
 * gdn_kv_write without a rotation, in one launch. Nothing else in the pool changes. No
 * two tokens of one call may have the same page and slot (the caller's contract; with
 * page_table_host and seq_lens_host a page that two requests write is GDN_ERR_ALIAS).
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE (E4M3 with FP32 io), GDN_ERR_RULE,
 * GDN_ERR_CAPACITY, GDN_ERR_ALIAS. */
int gdn_kv_write(const gdn_kv_params* params, const gdn_kv_tensors* tensors, const gdn_kv_cache* cache, void* stream);

/* Reads the tokens' keys and values from their pages into packed rows k and v
 * (E4M3 rows as code * 2^(s - 127), rounded to io where that is out of its range),
 * zeros where there is no page. With T_r = seq_lens[r] that is all a request has
 * cached. Errors as gdn_kv_write. */
int gdn_kv_read(const gdn_kv_params* params, const gdn_kv_tensors* tensors, const gdn_kv_cache* cache, void* stream);

/* ---- Attention over the cache. */
typedef struct gdn_attn_params {
  int32_t num_tokens;            /* N >= 0                                          */
  int32_t num_reqs;              /* R >= 0                                          */
  int32_t num_q_heads;           /* Hq: a multiple of the cache's Hk; query head h
                                    reads key head h / (Hq / Hk)                     */
  float scale;                   /* of q . k; <= 0 selects D^-1/2                   */
  int32_t window;                /* a token attends its newest `window` positions
                                    only; 0: all                                    */
  int32_t q_stride;              /* as in gdn_rope_params                           */
} gdn_attn_params;

typedef struct gdn_attn_tensors {
  const void* q;                 /* device, io [N, Hq, D], rows q_stride apart       */
  const int32_t* cu_seqlens;     /* as in gdn_kv_tensors                            */
  const int32_t* cu_seqlens_host;
  const int32_t* seq_lens;
  const int32_t* seq_lens_host;
  void* output;                  /* device, io [N, Hq, D]                           */
} gdn_attn_tensors;

/* out[n, h] = sum_p w_p v_p, w = softmax over the attended positions of
 * scale * q[n, h] . k_p. Token j of request r (position P = seq_lens[r] - T_r + j)
 * attends positions max(0, P - window + 1) .. P that have a page; a token that
 * attends none gives zeros. What the cache holds at other positions has no
 * influence, whatever it is. A row whose scores are all -inf gives zeros, too, and one
 * with a NaN score NaN. Scores, weights, sums and the output accumulate in FP32; FP16 io
 * takes the weights into the product with v to 2^-19 of each, or 2^-38 of the row's
 * largest (of weight times the value's scale with GDN_CACHE_E4M3).
 * Any number of tokens per request is taken; the kernels are made for decode and
 * verify, where the cache is read once for up to 32 rows (tokens x Hq / Hk) and, where
 * most requests have the same number of up to 256, mostly from the L2 for the rest.
 * Prompts are such segments of 32 rows, each of which walks the request's positions up
 * to its own from the first that any token of the call attends, so a long prompt is far
 * from the matrix cores' rate, and a window does not make it faster.
 * (N + R) Hq D / 64 is at most 2^30, else GDN_ERR_SHAPE.
 * The workspace (gdn_attn_workspace_bytes() bytes, disjoint from every tensor, 16-byte
 * aligned) needs no initial value; calls that overlap in time, and captured graphs
 * that may run at once, need one each.
 * Errors: GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_CAPACITY,
 * GDN_ERR_WORKSPACE, GDN_ERR_ALIAS. */
int gdn_attn_forward(const gdn_attn_params* params, const gdn_attn_tensors* tensors, const gdn_kv_cache* cache,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes gdn_attn_forward needs for these sizes, whatever the lengths
 * (the cache's pointers are not read). */
int gdn_attn_workspace_bytes(const gdn_attn_params* params, const gdn_kv_cache* cache, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H_ */

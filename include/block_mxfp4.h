/*
 * block_mxfp4.h - C ABI of the attention block around the 4-bit KV cache.
 *
 * What a decoder layer needs beside the MoE layer (moe_a16w4.h) and the cache
 * (kv_mxfp4.h), in the same format: a dense linear layer on MXFP4 weights with
 * bias, activation and residual in its epilogue, the position rotation of
 * queries and keys on the way into the quantising cache write, and attention of
 * a batch whose requests share a cached prefix.
 * Same library (libmoe_a16w4.so), same conventions as kv_mxfp4.h: device
 * pointers to caller-owned memory, work enqueued on ``stream``, MOE_OK or a
 * negative MOE_ERR_* code, argument checks before any CUDA call, nothing
 * allocated, no host synchronisation.  What a call writes may not share memory
 * with anything else that it is given (MOE_ERR_OVERLAP), but for the residual of
 * a linear layer.  The pages this library follows describe none of these
 * operators; they have no counterpart there.
 */
#ifndef BLOCK_MXFP4_H
#define BLOCK_MXFP4_H

#include "kv_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of a linear layer, on h = x W^T + bias (float32). */
#define LINEAR_ACT_NONE 0
#define LINEAR_ACT_SILU 1   /* h / (1 + exp(-h))                                        */
#define LINEAR_ACT_GELU 2   /* h (1 + erf(h / sqrt 2)) / 2                               */
#define LINEAR_ACT_SWIGLU 3 /* SiLU(h[:, :N/2]) * h[:, N/2:]: N/2 columns; the MoE's order */

/*
 * One linear layer.
 *   T  rows of x, 0 .. 2^24
 *   K  multiple of 32, 32 .. 65536
 *   N  rows of the weight, 1 .. 2^20 (even for SwiGLU), T * N at most 2^36
 *   act          LINEAR_ACT_*
 *   out_is_f32   0: bf16 results, 1: float32
 *   x_stride, res_stride, out_stride  elements between rows: x_stride a multiple
 *                of 8 and >= K, the others >= the columns of the result, all at most 2^38
 */
typedef struct linear_mxfp4 {
  int32_t T, K, N, act, out_is_f32;
  int64_t x_stride, res_stride, out_stride;
} linear_mxfp4_t;

/* Bytes of workspace that linear_a16w4_mxfp4 needs (256-byte aligned; 0 for
 * invalid sizes).  Its first 4 bytes are the status word, as in kv_mxfp4.h:
 * zero them, or call linear_mxfp4_read_status once; the rest does not matter.
 * It may be reused by calls ordered on one stream. */
size_t linear_mxfp4_workspace_bytes(const linear_mxfp4_t* d);

/*
 * out = act(x W^T + bias) + residual: products and sums in float32, rounded once.
 *   x         bf16 [T, K], 16-byte aligned
 *   w         uint8 [N, K/2]  E2M1 pairs, element 2j in the low nibble; 16-byte aligned
 *   w_scale   uint8 [N, K/32] E8M0, value 2^(s-127), 255 = NaN (a weight of 2^128 or
 *             more is infinite)
 *   bias      bf16 [N] or NULL
 *   residual  bf16 [T, columns] or NULL; may be ``out`` itself (same pointer and
 *             stride, bf16 results)
 *   out       bf16 or float32 [T, columns]; columns N, or N/2 for SwiGLU
 */
int linear_a16w4_mxfp4(const linear_mxfp4_t* d, const void* x, const uint8_t* w, const uint8_t* w_scale,
                       const void* bias, const void* residual, void* out, void* workspace, size_t workspace_bytes,
                       void* stream);

/* How a call of these sizes runs on the current device: 0, MMAs from registers; n >= 1, on
 * the tensor cores with K split in n (1: not split).  Or a negative MOE_ERR_* code. */
int linear_mxfp4_splits(const linear_mxfp4_t* d);

/* Copy the status word (MOE_STATUS_*) of a linear layer's workspace to *status and
 * clear it.  Synchronises ``stream``. */
int linear_mxfp4_read_status(void* workspace, uint32_t* status, void* stream);

/*
 * One step's rotation and cache write.
 *   N             tokens, 0 .. 2^24
 *   Hq            query heads, 0 (none) .. 16384
 *   x_is_f32      q, k, v: 0 bf16, 1 float32
 *   rotary_dim    leading elements of a head that are rotated, a multiple of 16 up to head_dim
 *   interleaved   0: pairs (i, i + rotary_dim / 2), 1: pairs (2i, 2i + 1)
 *   max_positions rows of cos_sin, >= 1
 *   position_offset  added to every position (>= 0): the length of a prefix that the requests share
 *   q_stride, k_stride, v_stride  elements between token rows: multiples of 16 bytes,
 *                 at least heads * head_dim
 */
typedef struct kv_mxfp4_rope {
  int32_t N, Hq, x_is_f32, rotary_dim, interleaved, max_positions, position_offset;
  int64_t q_stride, k_stride, v_stride;
} kv_mxfp4_rope_t;

/*
 * Rotate the queries and keys of N tokens by their positions, return the queries
 * and write keys and values, quantised (the rule of kv_mxfp4_append), to their slots.
 *   q, k, v     [N, Hq or num_kv_heads, head_dim], heads dense, pointers 16-byte aligned
 *               (slices of a fused projection); q and q_out are not looked at with Hq 0
 *   positions   int32 [N]; negative: padding, whose row of q_out is zeros and whose
 *               keys and values are not written.  A position past the table
 *               makes the token's queries and keys NaN.
 *   slots       int32 [N], as in kv_mxfp4_append
 *   cos_sin     float32 [max_positions, rotary_dim], 16-byte aligned: a position's
 *               rotary_dim / 2 cosines, then its sines
 *   q_out       bf16 [N, Hq, head_dim] dense, 16-byte aligned
 * A pair (a, b) becomes (a cos - b sin, b cos + a sin) in float32, both products and
 * the sum rounded; queries are then rounded to bf16, keys quantised.
 */
int kv_mxfp4_append_rope(const kv_mxfp4_cache_t* c, const kv_mxfp4_rope_t* r, const void* q, const void* k, const void* v,
                         const int32_t* positions, const int32_t* slots, const float* cos_sin, void* q_out, void* stream);

/*
 * Attention of a batch whose requests share a cached prefix, which is read once for
 * all of them.  The prefix has pages of its own, as has what each request holds
 * after it (so a request's own keys begin on a page of their own, numbered from 0).
 * It is for decoding batches behind a long prefix, from some 200,000 tokens of prefix times
 * requests on; below, and for prompts, kv_mxfp4_attention with the prefix's pages repeated
 * in every request's table takes as long or less.
 *   a              as in kv_mxfp4_attention; max_blocks, seq_lens, query_start and
 *                  positions are those of the requests' own tokens; window is 0
 *   shared_blocks  entries of shared_table, >= 1
 */

/* Bytes of workspace that kv_mxfp4_attention_shared needs (256-byte aligned; 0 for
 * invalid sizes): as kv_mxfp4_attention's, but it grows with N * Hq * head_dim (a
 * float32 sum of each row, for its own keys and for every slice of the prefix).  The
 * workspace of a call with more requests, rows or heads does for a smaller one too. */
size_t kv_mxfp4_attention_shared_workspace_bytes(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks);

/*
 * out = softmax over the prefix's keys and the request's own, as kv_mxfp4_attention
 * (its types, formulas, precision and status word: weights have 16 bits, in requests of
 * many rows, prompts, perhaps 11):
 *   shared_table  int32 [shared_blocks]  pages of the prefix; a page id outside the
 *                 cache makes its tokens invisible
 *   shared_len    int32 [1]  keys of the prefix (at most shared_blocks * page_size
 *                 are looked at, negative = none)
 *   block_table   int32 [R, max_blocks], seq_lens int32 [R]: the requests' own pages
 *                 and keys; every row sees the whole prefix, and its own keys as
 *                 without one.  Length 0: only the prefix.  A negative length: the
 *                 request sees nothing, not the prefix either (an empty place in the
 *                 batch: zeros, lse -inf, whatever its rows of q hold).
 *   query_start   int32 [R+1], not descending
 * The rest as in kv_mxfp4_attention.
 */
int kv_mxfp4_attention_shared(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks, const void* q,
                              const int32_t* shared_table, const int32_t* shared_len, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* query_start, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream);

/* How a call of these sizes runs: 0, the prefix is streamed; n >= 1, on the tensor cores, cut into
 * n slices (fewer where the workspace is one of a larger batch).  Or a negative MOE_ERR_* code. */
int kv_mxfp4_attention_shared_slices(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_MXFP4_H */

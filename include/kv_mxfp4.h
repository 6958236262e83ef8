/*
 * kv_mxfp4.h - C ABI of the 4-bit KV cache and the attention that reads it.
 *
 * The attention half of a decoder layer, next to the MoE layer of
 * moe_a16w4.h: a paged key/value cache held in MXFP4 (packed E2M1 nibbles, one
 * E8M0 scale byte per 32 values of a head's row, the rule of
 * moe_quantize_act), page tables and slot maps built on the GPU from request
 * lengths, the quantising write, a read-back, and attention over the cache.
 * Same library (libmoe_a16w4.so), same conventions as moe_a16w4.h: device
 * pointers to caller-owned memory, work enqueued on ``stream``, MOE_OK or a
 * negative MOE_ERR_* code, argument checks before any CUDA call, nothing
 * allocated, no host synchronisation.  What a call writes may not share memory
 * with anything else that it is given (MOE_ERR_OVERLAP).  The pages this library follows
 * describe no cache; these operators have no counterpart there.
 */
#ifndef KV_MXFP4_H
#define KV_MXFP4_H

#include "moe_a16w4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One layer's cache: uint8 [num_pages, num_kv_heads, page_size / 16, 17 * head_dim].
 * A slot is page * page_size + offset.  Each record holds 16 consecutive
 * tokens of one head in the order in which the lanes of an m16n8k16 MMA take
 * their operands.  With NB = head_dim / 32 scale blocks per row, and byte j of
 * a row holding elements 2j (low nibble) and 2j + 1:
 *   K codes  [half 2][g 8][t 4][NB][4]      token 8 half + g, row byte 16 b + 4 t + j
 *   V codes  [hi 2][g 8][t 4][lo 2][NB][2]  token 8 hi + 2 t + lo, row byte 16 b + 2 g + j
 *   K scales [16][NB], V scales [16][NB]    value code * 2^(scale - 127), 255 = NaN
 *   data          16-byte aligned
 *   num_pages     >= 1, num_pages * page_size <= 2^31 - 1
 *   page_size     16, 32, 64, 128 or 256 tokens
 *   num_kv_heads  1 .. 256
 *   head_dim      64 or 128
 * Slots that were never written may hold anything: no call reads them unless
 * a slot map or a request length says they are live.
 */
typedef struct kv_mxfp4_cache {
  void* data;
  int32_t num_pages, page_size, num_kv_heads, head_dim;
} kv_mxfp4_cache_t;

/* Bytes of a cache (data is not looked at); 0 if a size is outside its set. */
size_t kv_mxfp4_cache_bytes(const kv_mxfp4_cache_t* c);

/*
 * Page tables and slot maps of one step, from request lengths.
 *   R              requests, 0 .. 8192
 *   page_size      as the cache's
 *   max_blocks     columns of block_table, >= 1
 *   max_tokens     entries of slots and positions, >= 0
 *   ring_size      entries of free_ring, >= 1
 *   cached_lens    int32 [R]  tokens a request has in the cache (>= 0)
 *   new_lens       int32 [R]  tokens it adds in this step (>= 0), or -1: the
 *                  request is finished and gives its pages back
 *   block_table    int32 [R, max_blocks], row stride max_blocks; the first
 *                  ceil(cached / page_size) entries of a row are its pages.
 *                  The entries of new pages are written; others stay.
 *   free_ring      int32 [ring_size]  ring of free page ids; pages are taken
 *                  from its head in request order and given back at its end
 *   ring_state     int32 [2]  {head, free pages}
 *   seq_lens       int32 [R]  cached + new; 0 for a finished request; -1 for a
 *                  request that is refused: its tokens do not fit in
 *                  max_tokens, its pages not in its row, it would hold more
 *                  than 2^31 - 1 tokens, or the free pages do
 *                  not last (pages given back in the same call are not taken;
 *                  a refused request's pages are counted for those after it
 *                  only where it was refused for want of free pages, so one
 *                  that needs a page is then refused too)
 *   query_start    int32 [R+1]  exclusive sum of max(new, 0), refused ones too
 *   slots          int32 [max_tokens]  cache slot of each new token; -1 for
 *                  tokens of refused requests and past query_start[R]
 *   positions      int32 [max_tokens]  position of each new token in its
 *                  request (at most 2^31 - 1); -1 past query_start[R]
 *   ring_state_out int32 [2]  the ring afterwards
 * block_table and free_ring count as written.  Lengths are not updated in place:
 * copy seq_lens over cached_lens after the call, but for -1.
 * Everything but block_table and free_ring is written whole; with the same
 * inputs a second call writes the same again.
 */
int kv_mxfp4_page_tables(int32_t R, int32_t page_size, int32_t max_blocks, int32_t max_tokens, int32_t ring_size,
                         const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table, int32_t* free_ring,
                         const int32_t* ring_state, int32_t* seq_lens, int32_t* query_start, int32_t* slots,
                         int32_t* positions, int32_t* ring_state_out, void* stream);

/*
 * Quantise the rows of N new tokens and write them to their slots.
 *   k, v      [N, num_kv_heads, head_dim], bf16 (x_is_f32 = 0) or float32 (1):
 *             heads dense, token rows k_stride / v_stride elements apart (a
 *             slice of a fused projection); pointers 16-byte aligned, strides
 *             multiples of 16 bytes and at least num_kv_heads * head_dim
 *   slots     int32 [N]; a slot outside the cache (-1) writes nothing.  No
 *             slot may occur twice.
 * Rule per 32 values: the MOE_AQ_MXFP4 rule of moe_quantize_act; beyond its
 * contract, a block with a NaN gets scale byte 255, infinities saturate (scale
 * byte 252, code +-6).
 */
int kv_mxfp4_append(const kv_mxfp4_cache_t* c, const void* k, const void* v, int32_t x_is_f32, int64_t k_stride,
                    int64_t v_stride, int32_t N, const int32_t* slots, void* stream);

/*
 * Read N tokens back: the values their slots hold, exact in bf16 (infinite
 * where code * 2^(scale - 127) overflows, NaN in a block of scale byte 255).
 *   k_out, v_out  bf16 [N, num_kv_heads, head_dim] dense, 16-byte aligned;
 *                 zeros for a slot outside the cache
 */
int kv_mxfp4_gather(const kv_mxfp4_cache_t* c, const int32_t* slots, int32_t N, void* k_out, void* v_out,
                    void* stream);

/*
 * One attention call.
 *   R           requests, 0 .. 65535
 *   N           query rows (tokens) in q and out, 0 .. 2^24
 *   Hq          query heads, a multiple of num_kv_heads, at most 64 per kv head
 *   max_blocks  columns of block_table
 *   max_q_len   largest query_start[r+1] - query_start[r]; longer requests'
 *               further rows are left unwritten
 *   causal      1: row i of a request of q rows and length n sits at position
 *               n - q + i and sees keys up to it; 0: it sees all n keys
 *   window      0: off; w > 0 (causal only): only the w keys up to its position
 *   q_stride    elements between the rows of q (multiple of 8, >= Hq * head_dim)
 *   scale       factor of q.k, finite
 */
typedef struct kv_mxfp4_attn {
  int32_t R, N, Hq, max_blocks, max_q_len;
  int32_t causal, window;
  int64_t q_stride;
  float scale;
} kv_mxfp4_attn_t;

/* Bytes of workspace that kv_mxfp4_attention needs (256-byte aligned; 0 for
 * invalid sizes).  It may be reused by calls ordered on one stream; its
 * contents do not matter, but its first 4 bytes, the status word, read back
 * what the memory held until cleared (zero them, or call
 * kv_mxfp4_read_status once). */
size_t kv_mxfp4_attention_workspace_bytes(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a);

/*
 * Attention over the cache:
 *   S = scale * q . k_j, out = sum_j softmax(S)_j v_j over the visible keys
 *   q            bf16 [N, Hq, head_dim], 16-byte aligned; query head h reads kv
 *                head h / (Hq / num_kv_heads)
 *   block_table  int32 [R, max_blocks]; a page id outside the cache makes its
 *                tokens invisible
 *   seq_lens     int32 [R]  keys of each request, new tokens included (at most
 *                max_blocks * page_size are looked at, negative = none)
 *   query_start  int32 [R+1]  first row of each request
 *   out          bf16 [N, Hq, head_dim] dense, 16-byte aligned
 *   lse          float32 [N, Hq] or NULL: ln sum exp S
 * A row that sees no key gets zeros (lse -inf).  Scores, softmax statistics
 * and sums are float32; scales of any size are honoured.  Elements of q below 2^-31
 * of their row's largest may lose bits, where that moves no score by more than
 * 2^-16 (units of log2).  The weights exp(S - m) enter their product with 16 bits
 * down to 2^-126; those of a row that sees more than 256 positions, in a request of
 * many rows (a prompt), may have 11 bits, below 2^-23 of the row's largest multiples
 * of 2^-33 of it.  A token with a scale byte 255 in its K or V row counts as NaN as a
 * whole: rows that see it are NaN.  So are rows of q with an infinite or NaN element
 * that see a key.
 * Rows outside every request are left unwritten.
 */
int kv_mxfp4_attention(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, const void* q, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* query_start, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Copy the status word (MOE_STATUS_*) of an attention workspace to *status and
 * clear it.  Synchronises ``stream``. */
int kv_mxfp4_read_status(void* workspace, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KV_MXFP4_H */

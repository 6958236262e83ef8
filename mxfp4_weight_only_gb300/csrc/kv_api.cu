// C ABI entry points of the 4-bit KV cache: argument checks and dispatch.
#include "kv_checks.h"

using namespace moe;

extern "C" {

size_t kv_mxfp4_cache_bytes(const kv_mxfp4_cache_t* c) {
  if (!cache_valid(c)) return 0;
  return (size_t)c->num_pages * c->num_kv_heads * (c->page_size / kKvGroup) * kv_record_bytes(c->head_dim);
}

int kv_mxfp4_page_tables(int32_t R, int32_t page_size, int32_t max_blocks, int32_t max_tokens, int32_t ring_size,
                         const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table, int32_t* free_ring,
                         const int32_t* ring_state, int32_t* seq_lens, int32_t* query_start, int32_t* slots,
                         int32_t* positions, int32_t* ring_state_out, void* stream) {
  const int shift = shift_of(page_size);
  if (R < 0 || R > kMaxTableRequests || shift < 0 || max_blocks < 1 || max_tokens < 0 || ring_size < 1)
    return MOE_ERR_BAD_DIMS;
  if (!free_ring || !ring_state || !query_start || !ring_state_out) return MOE_ERR_NULL;
  if (R > 0 && (!cached_lens || !new_lens || !block_table || !seq_lens)) return MOE_ERR_NULL;
  if (max_tokens > 0 && (!slots || !positions)) return MOE_ERR_NULL;
  const void* all[] = {cached_lens, new_lens, block_table, free_ring, ring_state, seq_lens, query_start, slots, positions, ring_state_out};
  for (const void* p : all)
    if (!aligned(p, 4)) return MOE_ERR_ALIGN;
  // Every CTA of the launch reads the lengths and the ring's state, the block
  // table and the ring while others write their outputs: none may share memory.
  const uint64_t r4 = 4ull * (uint64_t)R, t4 = 4ull * (uint64_t)max_tokens;
  const Span span[] = {{cached_lens, r4}, {new_lens, r4}, {ring_state, 8},  // read
                       {block_table, r4 * (uint64_t)max_blocks}, {free_ring, 4ull * (uint64_t)ring_size},
                       {seq_lens, r4}, {query_start, r4 + 4}, {slots, t4}, {positions, t4}, {ring_state_out, 8}};
  if (any_overlap(span, 3)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  const PageTableArgs a{R, shift, max_blocks, max_tokens, ring_size, cached_lens, new_lens, block_table, free_ring,
                        ring_state, seq_lens, query_start, slots, positions, ring_state_out};
  return launch_page_tables(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int kv_mxfp4_append(const kv_mxfp4_cache_t* c, const void* k, const void* v, int32_t x_is_f32, int64_t k_stride,
                    int64_t v_stride, int32_t N, const int32_t* slots, void* stream) {
  if (!c) return MOE_ERR_NULL;
  if (!cache_valid(c) || N < 0 || N > (1 << 24) || (x_is_f32 != 0 && x_is_f32 != 1)) return MOE_ERR_BAD_DIMS;
  const int64_t row = (int64_t)c->num_kv_heads * c->head_dim, unit = x_is_f32 ? 4 : 8;
  if (k_stride < row || v_stride < row || k_stride % unit || v_stride % unit || k_stride > (1ll << 40) ||
      v_stride > (1ll << 40))
    return MOE_ERR_BAD_DIMS;
  if (N == 0) return MOE_OK;
  if (!c->data || !k || !v || !slots) return MOE_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return MOE_ERR_ALIGN;
  const uint64_t size = x_is_f32 ? 4 : 2, n1 = (uint64_t)N - 1;
  const Span span[] = {{k, size * (n1 * (uint64_t)k_stride + (uint64_t)row)}, {v, size * (n1 * (uint64_t)v_stride + (uint64_t)row)},
                       {slots, 4ull * (uint64_t)N}, {c->data, kv_mxfp4_cache_bytes(c)}};
  if (any_overlap(span, 3)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  return launch_kv_append(view_of(c), k, v, x_is_f32 == 1, k_stride, v_stride, N, slots, sms,
                          reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int kv_mxfp4_gather(const kv_mxfp4_cache_t* c, const int32_t* slots, int32_t N, void* k_out, void* v_out,
                    void* stream) {
  if (!c) return MOE_ERR_NULL;
  if (!cache_valid(c) || N < 0 || N > (1 << 24)) return MOE_ERR_BAD_DIMS;
  if (N == 0) return MOE_OK;
  if (!c->data || !slots || !k_out || !v_out) return MOE_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 4)) return MOE_ERR_ALIGN;
  const uint64_t rows = 2ull * (uint64_t)N * (uint64_t)c->num_kv_heads * (uint64_t)c->head_dim;
  const Span span[] = {{slots, 4ull * (uint64_t)N}, {c->data, kv_mxfp4_cache_bytes(c)}, {k_out, rows}, {v_out, rows}};
  if (any_overlap(span, 2)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  return launch_kv_gather(view_of(c), slots, N, k_out, v_out, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

size_t kv_mxfp4_attention_workspace_bytes(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a) {
  if (!cache_valid(c) || !a || !attn_valid(c, a)) return 0;
  return kv_attention_workspace(view_of(c), a);
}

int kv_mxfp4_attention(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, const void* q, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* query_start, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const WaitSettings wait = take_wait_settings();  // the hook applies to this call only
  if (!c || !a) return MOE_ERR_NULL;
  if (!cache_valid(c) || !attn_valid(c, a)) return MOE_ERR_BAD_DIMS;
  if (a->R == 0 || a->N == 0 || a->max_q_len == 0) return MOE_OK;
  if (!c->data || !q || !block_table || !seq_lens || !query_start || !out || !workspace) return MOE_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(lse, 4))
    return MOE_ERR_ALIGN;
  const KvView view = view_of(c);
  const size_t need = kv_attention_workspace(view, a);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  // q is read again after rows of out have been written (by the streaming kernel, for marked prompts)
  const uint64_t heads = (uint64_t)a->N * (uint64_t)a->Hq, D = (uint64_t)c->head_dim;
  const Span span[] = {{q, 2 * ((uint64_t)(a->N - 1) * (uint64_t)a->q_stride + (uint64_t)a->Hq * D)},
                       {block_table, 4ull * (uint64_t)a->R * (uint64_t)a->max_blocks}, {seq_lens, 4ull * (uint64_t)a->R},
                       {query_start, 4ull * (uint64_t)a->R + 4}, {c->data, kv_mxfp4_cache_bytes(c)},
                       {out, 2 * heads * D}, {lse, lse ? 4 * heads : 0}, {workspace, need}};
  if (any_overlap(span, 5)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  const KvAttnArgs g = attn_args(view, a, q, block_table, seq_lens, query_start, out, lse, workspace, sms, wait);
  return launch_kv_attention(g, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int kv_mxfp4_read_status(void* workspace, uint32_t* status, void* stream) {
  if (!workspace || !status) return MOE_ERR_NULL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, workspace, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(workspace, 0, sizeof(v), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  *status = v;
  return MOE_OK;
}

}  // extern "C"

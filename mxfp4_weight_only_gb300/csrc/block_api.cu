// C ABI entry points of the attention block: argument checks and dispatch.
#include "kv_checks.h"
#include "linear.cuh"

using namespace moe;

namespace {

constexpr size_t kLinearWorkspace = 256;  // the status word

bool linear_valid(const linear_mxfp4_t* d) {
  if (d->T < 0 || d->T > (1 << 24) || d->K < 32 || d->K > 65536 || d->K % 32 || d->N < 1 || d->N > (1 << 20)) return false;
  if (d->act < LINEAR_ACT_NONE || d->act > LINEAR_ACT_SWIGLU || (d->out_is_f32 != 0 && d->out_is_f32 != 1)) return false;
  if (d->act == LINEAR_ACT_SWIGLU && d->N % 2) return false;
  if ((long long)d->T * d->N > 1ll << 36) return false;
  const int64_t cols = d->act == LINEAR_ACT_SWIGLU ? d->N / 2 : d->N, most = 1ll << 38;  // (tensor maps: strides below 2^40 bytes)
  return d->x_stride % 8 == 0 && d->x_stride >= d->K && d->x_stride <= most && d->res_stride >= cols &&
         d->res_stride <= most && d->out_stride >= cols && d->out_stride <= most;
}

// The sizes of a call on a device of ``sms`` SMs.
LinearArgs linear_sizes(const linear_mxfp4_t* d, int sms) {
  LinearArgs a{};
  a.T = d->T; a.K = d->K; a.N = d->N; a.act = d->act; a.f32 = d->out_is_f32 == 1;
  a.cols = d->act == LINEAR_ACT_SWIGLU ? d->N / 2 : d->N;
  a.x_stride = d->x_stride; a.res_stride = d->res_stride; a.out_stride = d->out_stride;
  a.num_sms = sms;
  return a;
}

bool shared_valid(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t blocks) {
  return cache_valid(c) && a && attn_valid(c, a) && a->window == 0 && blocks >= 1 &&
         (long long)blocks * c->page_size <= 0x7FFFFFFFll;
}

}  // namespace

extern "C" {

size_t linear_mxfp4_workspace_bytes(const linear_mxfp4_t* d) { return d && linear_valid(d) ? kLinearWorkspace : 0; }

int linear_a16w4_mxfp4(const linear_mxfp4_t* d, const void* x, const uint8_t* w, const uint8_t* w_scale, const void* bias,
                       const void* residual, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  const WaitSettings wait = take_wait_settings();  // the hook applies to this call only
  if (!d) return MOE_ERR_NULL;
  if (!linear_valid(d)) return MOE_ERR_BAD_DIMS;
  if (d->T == 0) return MOE_OK;
  if (!x || !w || !w_scale || !out || !workspace) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 2) || !aligned(residual, 2) ||
      !aligned(out, d->out_is_f32 ? 4 : 2) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < kLinearWorkspace) return MOE_ERR_WORKSPACE;
  const uint64_t cols = d->act == LINEAR_ACT_SWIGLU ? d->N / 2 : d->N, n1 = (uint64_t)d->T - 1, N = (uint64_t)d->N;
  // each value of a residual that is ``out`` itself is read by the thread that writes it
  const bool in_place = residual == out && !d->out_is_f32 && d->res_stride == d->out_stride;
  const Span span[] = {{x, 2 * (n1 * (uint64_t)d->x_stride + (uint64_t)d->K)}, {w, N * (uint64_t)d->K / 2},
                       {w_scale, N * (uint64_t)d->K / 32}, {bias, bias ? 2 * N : 0},
                       {residual, residual && !in_place ? 2 * (n1 * (uint64_t)d->res_stride + cols) : 0},
                       {out, (d->out_is_f32 ? 4 : 2) * (n1 * (uint64_t)d->out_stride + cols)},
                       {workspace, kLinearWorkspace}};
  if (any_overlap(span, 5)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  LinearArgs a = linear_sizes(d, sms);
  a.x = reinterpret_cast<const uint16_t*>(x);
  a.w = w; a.ws = w_scale;
  a.bias = reinterpret_cast<const uint16_t*>(bias);
  a.res = reinterpret_cast<const uint16_t*>(residual);
  a.out = out;
  a.status = reinterpret_cast<uint32_t*>(workspace);
  a.wait = wait;
  return launch_linear(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int linear_mxfp4_splits(const linear_mxfp4_t* d) {
  if (!d) return MOE_ERR_NULL;
  if (!linear_valid(d)) return MOE_ERR_BAD_DIMS;
  int sms = 0, splits = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  return linear_splits(linear_sizes(d, sms), &splits) == cudaSuccess ? splits : MOE_ERR_CUDA;
}

int linear_mxfp4_read_status(void* workspace, uint32_t* status, void* stream) {
  return kv_mxfp4_read_status(workspace, status, stream);
}

int kv_mxfp4_append_rope(const kv_mxfp4_cache_t* c, const kv_mxfp4_rope_t* r, const void* q, const void* k, const void* v,
                         const int32_t* positions, const int32_t* slots, const float* cos_sin, void* q_out, void* stream) {
  if (!c || !r) return MOE_ERR_NULL;
  if (!cache_valid(c) || r->N < 0 || r->N > (1 << 24) || r->Hq < 0 || r->Hq > 16384 ||
      (r->x_is_f32 != 0 && r->x_is_f32 != 1) || r->rotary_dim < 16 || r->rotary_dim > c->head_dim || r->rotary_dim % 16 ||
      (r->interleaved != 0 && r->interleaved != 1) || r->max_positions < 1 || r->position_offset < 0)
    return MOE_ERR_BAD_DIMS;
  const int64_t row = (int64_t)c->num_kv_heads * c->head_dim, q_row = (int64_t)r->Hq * c->head_dim;
  const int64_t unit = r->x_is_f32 ? 4 : 8, most = 1ll << 40;
  auto stride_ok = [&](int64_t s, int64_t least) { return s >= least && s % unit == 0 && s <= most; };
  if (!stride_ok(r->k_stride, row) || !stride_ok(r->v_stride, row) || (r->Hq && !stride_ok(r->q_stride, q_row)))
    return MOE_ERR_BAD_DIMS;
  if (r->N == 0) return MOE_OK;
  if (!c->data || !k || !v || !positions || !slots || !cos_sin || (r->Hq && (!q || !q_out))) return MOE_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(positions, 4) || !aligned(slots, 4) ||
      !aligned(cos_sin, 16) || (r->Hq && (!aligned(q, 16) || !aligned(q_out, 16))))
    return MOE_ERR_ALIGN;
  const uint64_t size = r->x_is_f32 ? 4 : 2, n1 = (uint64_t)r->N - 1, N = (uint64_t)r->N;
  const Span span[] = {{k, size * (n1 * (uint64_t)r->k_stride + (uint64_t)row)}, {v, size * (n1 * (uint64_t)r->v_stride + (uint64_t)row)},
                       {q, r->Hq ? size * (n1 * (uint64_t)r->q_stride + (uint64_t)q_row) : 0}, {positions, 4 * N}, {slots, 4 * N},
                       {cos_sin, 4ull * (uint64_t)r->max_positions * (uint64_t)r->rotary_dim},
                       {c->data, kv_mxfp4_cache_bytes(c)}, {q_out, r->Hq ? 2 * N * (uint64_t)q_row : 0}};
  if (any_overlap(span, 6)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  const RopeArgs a{r->N, r->Hq, r->rotary_dim, r->max_positions, r->position_offset, r->q_stride, r->k_stride, r->v_stride,
                   q, k, v, positions, slots, cos_sin, reinterpret_cast<uint16_t*>(q_out)};
  return launch_kv_append_rope(view_of(c), a, r->x_is_f32 == 1, r->interleaved == 1, sms,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

size_t kv_mxfp4_attention_shared_workspace_bytes(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks) {
  if (!shared_valid(c, a, shared_blocks)) return 0;
  const KvView view = view_of(c);
  return kv_shared_workspace(view, a, kv_shared_plan(view, a, shared_blocks).splits);
}

int kv_mxfp4_attention_shared(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks, const void* q,
                              const int32_t* shared_table, const int32_t* shared_len, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* query_start, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const WaitSettings wait = take_wait_settings();  // the hook applies to this call only
  if (!c || !a) return MOE_ERR_NULL;
  if (!shared_valid(c, a, shared_blocks)) return MOE_ERR_BAD_DIMS;
  if (a->R == 0 || a->N == 0 || a->max_q_len == 0) return MOE_OK;
  if (!c->data || !q || !shared_table || !shared_len || !block_table || !seq_lens || !query_start || !out || !workspace)
    return MOE_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(shared_table, 4) || !aligned(shared_len, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(query_start, 4) || !aligned(lse, 4))
    return MOE_ERR_ALIGN;
  const KvView view = view_of(c);
  // fewer rows may be cut into more slices: a workspace for more rows does, with fewer of them
  const KvSharedPlan plan = kv_shared_plan(view, a, shared_blocks);
  int splits = plan.splits;
  while (splits > 1 && kv_shared_workspace(view, a, splits) > workspace_bytes) --splits;
  const size_t need = kv_shared_workspace(view, a, splits);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  const uint64_t heads = (uint64_t)a->N * (uint64_t)a->Hq, D = (uint64_t)c->head_dim, R = (uint64_t)a->R;
  const Span span[] = {{q, 2 * ((uint64_t)(a->N - 1) * (uint64_t)a->q_stride + (uint64_t)a->Hq * D)},
                       {shared_table, 4ull * (uint64_t)shared_blocks}, {shared_len, 4},
                       {block_table, 4 * R * (uint64_t)a->max_blocks}, {seq_lens, 4 * R}, {query_start, 4 * R + 4},
                       {c->data, kv_mxfp4_cache_bytes(c)}, {out, 2 * heads * D}, {lse, lse ? 4 * heads : 0}, {workspace, need}};
  if (any_overlap(span, 7)) return MOE_ERR_OVERLAP;
  int sms = 0;
  const int rc = check_device(&sms);
  if (rc != MOE_OK) return rc;
  KvAttnArgs g = attn_args(view, a, q, block_table, seq_lens, query_start, out, lse, workspace, sms, wait);
  g.sh.splits = splits;
  g.sh.row_limit = plan.stream ? INT32_MAX : 0;
  g.sh.blocks = shared_blocks;
  g.sh.table = shared_table;
  g.sh.len = shared_len;
  return launch_kv_shared(g, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int kv_mxfp4_attention_shared_slices(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a, int32_t shared_blocks) {
  if (!c || !a) return MOE_ERR_NULL;
  if (!shared_valid(c, a, shared_blocks)) return MOE_ERR_BAD_DIMS;
  const KvSharedPlan plan = kv_shared_plan(view_of(c), a, shared_blocks);
  return plan.stream ? 0 : plan.splits;
}

}  // extern "C"

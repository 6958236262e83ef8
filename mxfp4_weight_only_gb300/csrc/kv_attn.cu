// Attention over the 4-bit KV cache (kv_mxfp4_attention): workspace and choice of kernels.
#include "kv_internal.h"

namespace moe {

namespace {
constexpr size_t kStatusBytes = 256;  // the status word leads every workspace
}

size_t kv_attention_workspace(const KvView& c, const kv_mxfp4_attn_t*) {
  return kStatusBytes + kv_stream_workspace(c.D);
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.cache.heads;
  const long long rows = (long long)a.max_q_len * G;
  return launch_kv_stream(a, 0x7FFFFFFF, rows <= 8 ? 1 : 2, a.workspace + kStatusBytes, s);
}

}  // namespace moe

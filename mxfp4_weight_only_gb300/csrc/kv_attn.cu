// Attention over the 4-bit KV cache (kv_mxfp4_attention): workspace and choice of kernels.
#include "kv_internal.h"

namespace moe {

namespace {
constexpr size_t kStatusBytes = 256;  // the status word leads every workspace
// Requests of up to this many rows (query tokens x query heads per kv head) are
// streamed; longer ones go to the tensor-core kernel.
constexpr int kStreamRows = 64;
}

size_t kv_attention_workspace(const KvView& c, const kv_mxfp4_attn_t* a) {
  return kStatusBytes + ((kv_stream_workspace(c.D) + 255) & ~size_t(255)) + sizeof(int32_t) * (size_t)a->R;
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.cache.heads;
  const long long rows = (long long)a.max_q_len * G;
  uint8_t* ws = a.workspace + kStatusBytes;
  if (rows <= kStreamRows) return launch_kv_stream(a, kStreamRows, nullptr, rows <= 8 ? 1 : 2, ws, s);
  int32_t* odd = reinterpret_cast<int32_t*>(ws + ((kv_stream_workspace(a.cache.D) + 255) & ~size_t(255)));
  const cudaError_t e = launch_kv_prompt(a, kStreamRows, odd, s);
  if (e != cudaSuccess) return e;
  return launch_kv_stream(a, kStreamRows, odd, G <= 8 ? 1 : 2, ws, s);
}

}  // namespace moe

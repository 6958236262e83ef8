// Attention over the 4-bit KV cache (kv_mxfp4_attention): workspace and choice of kernels.
#include <algorithm>

#include "kv_internal.h"

namespace moe {

namespace {
constexpr size_t kStatusBytes = 256;  // the status word leads every workspace
}  // namespace

// Requests of up to this many rows (query tokens x query heads per kv head) are
// streamed, longer ones go to the tensor-core kernel.  A CTA of that one, up to
// 256 rows of a request and kv head, takes 15 to 17 ns a key and does not split the
// keys; the streaming kernel shares all work between the SMs and takes 6.5 ns a
// key, SM and 16 rows.  With at least a request and head per SM the tensor cores
// win above 2 tiles of 16 (32 requests x 8 heads x 8192 keys: 32 rows 200 us
// streamed, 249 there; 48 rows 294 and 250); with fewer, other SMs help the
// streaming kernel only (4 x 8 x 32768: 128 rows 381 and 478 us, 192 rows 563 and 524).
int kv_stream_rows(const KvAttnArgs& a) {
  const long long pairs = (long long)a.R * a.cache.heads;
  return 16 * (int)std::max<long long>(2, 23LL * a.num_sms / (10 * std::max<long long>(pairs, 1)));
}

size_t kv_attention_workspace(const KvView& c, const kv_mxfp4_attn_t* a) {
  return kStatusBytes + ((kv_stream_workspace(c.D) + 255) & ~size_t(255)) + sizeof(int32_t) * (size_t)a->R;
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.cache.heads;
  const long long rows = (long long)a.max_q_len * G;
  uint8_t* ws = a.workspace + kStatusBytes;
  const int limit = kv_stream_rows(a);
  // row tiles of 8 where they hold all rows, else of 16 (32 requests x 8 heads x 4096
  // keys: 8 rows 44 us in a tile of 8, 62 in one of 16; 16 rows 74 and 63)
  if (rows <= limit) return launch_kv_stream(a, limit, nullptr, rows <= 8 ? 1 : 2, ws, s);
  int32_t* odd = reinterpret_cast<int32_t*>(ws + ((kv_stream_workspace(a.cache.D) + 255) & ~size_t(255)));
  const cudaError_t e = launch_kv_prompt(a, limit, odd, s);
  if (e != cudaSuccess) return e;
  // (beside prompts, a decoding request has G rows)
  return launch_kv_stream(a, limit, odd, G <= 8 ? 1 : 2, ws, s);
}

}  // namespace moe

// Argument checks shared by the C ABI entry points of the 4-bit cache and of the attention block.
#pragma once

#include <math.h>

#include "kv_internal.h"

namespace moe {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device check and SM count, once per device and host thread (two attribute
// queries a call weigh on calls of a few microseconds).
inline int check_device(int* num_sms) {
  thread_local int known = -1, sms = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev != known) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (major != 10 || minor != 3) return MOE_ERR_DEVICE;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MOE_ERR_CUDA;
    known = dev;
  }
  *num_sms = sms;
  return MOE_OK;
}

// Do ``na`` bytes at a and ``nb`` bytes at b share one?
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < na : x - y < nb;
}

struct Span {
  const void* p;
  uint64_t bytes;
};
// Does one of the spans from ``first`` on (the written ones) share memory with any span before it?
template <int N>
inline bool any_overlap(const Span (&s)[N], int first) {
  for (int i = first; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (s[i].bytes && s[j].bytes && overlap(s[i].p, s[i].bytes, s[j].p, s[j].bytes)) return true;
  return false;
}

inline int shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

inline bool cache_valid(const kv_mxfp4_cache_t* c) {
  return c && shift_of(c->page_size) > 0 && c->num_pages >= 1 &&
         (long long)c->num_pages * c->page_size <= 0x7FFFFFFFll && c->num_kv_heads >= 1 && c->num_kv_heads <= 256 &&
         (c->head_dim == 64 || c->head_dim == 128);
}

inline KvView view_of(const kv_mxfp4_cache_t* c) {
  return KvView{reinterpret_cast<uint8_t*>(c->data), c->num_pages, shift_of(c->page_size), c->num_kv_heads, c->head_dim};
}

inline bool attn_valid(const kv_mxfp4_cache_t* c, const kv_mxfp4_attn_t* a) {
  if (a->R < 0 || a->R > 65535 || a->N < 0 || a->N > (1 << 24)) return false;
  if (a->Hq < 1 || a->Hq % c->num_kv_heads || a->Hq / c->num_kv_heads > 64) return false;
  if (a->max_blocks < 1 || (long long)a->max_blocks * c->page_size > 0x7FFFFFFFll) return false;
  if (a->max_q_len < 0 || (a->causal != 0 && a->causal != 1)) return false;
  if (a->window < 0 || (a->window > 0 && !a->causal)) return false;
  if (a->q_stride % 8 || a->q_stride < (long long)a->Hq * c->head_dim || a->q_stride > (1ll << 40)) return false;
  return isfinite(a->scale);
}

inline KvAttnArgs attn_args(const KvView& view, const kv_mxfp4_attn_t* a, const void* q, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* query_start, void* out, float* lse, void* workspace,
                            int sms, const WaitSettings& wait) {
  KvAttnArgs g{};
  g.cache = view;
  g.R = a->R; g.N = a->N; g.Hq = a->Hq; g.max_blocks = a->max_blocks; g.max_q_len = a->max_q_len;
  g.causal = a->causal; g.window = a->window; g.q_stride = a->q_stride; g.scale = a->scale;
  g.q = reinterpret_cast<const uint16_t*>(q);
  g.table = block_table; g.seq_lens = seq_lens; g.query_start = query_start;
  g.out = reinterpret_cast<uint16_t*>(out);
  g.lse = lse;
  g.workspace = reinterpret_cast<uint8_t*>(workspace);
  g.status = reinterpret_cast<uint32_t*>(workspace);
  g.num_sms = sms;
  g.wait = wait;
  return g;
}

}  // namespace moe

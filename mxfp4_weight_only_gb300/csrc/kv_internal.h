// Internal declarations of the 4-bit KV cache operators.
#pragma once

#include <atomic>

#include "../../include/kv_mxfp4.h"
#include "moe_internal.h"
#ifdef __CUDACC__
#include "common.cuh"
#endif

namespace moe {

// Lets ``kern`` use ``bytes`` of dynamic shared memory: asked of the runtime once
// per device (``done``: one bit per device, a static of the caller's).
template <typename K>
inline cudaError_t allow_shared(K kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

#ifdef __CUDACC__
// mbar_wait by a whole warp, with one result: lanes run out of time (or see the
// abort flag) one by one, and those that went on would wait in the next
// collective for those that left.  ``abort`` (may be null): a flag of the CTA
// that ends a wait in progress.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint32_t* status, uint64_t limit_ns,
                                               const volatile int* abort = nullptr) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 15u) == 15u && abort && __any_sync(0xffffffffu, *abort != 0)) return false;
    if ((i & 255u) == 255u && __any_sync(0xffffffffu, global_ns() - t0 > limit_ns)) {
      atomicOr(status, kStatusWaitTimeout);
      return false;
    }
  }
}
#endif

// A record: 16 tokens of one kv head (see kv_mxfp4_cache_t for its layout).
constexpr int kKvGroup = 16;
__host__ __device__ constexpr int kv_record_bytes(int D) { return 17 * D; }

// Device view of a cache.
struct KvView {
  uint8_t* data;
  int num_pages, page_shift, heads, D;
  // record of token group ``gi`` (16 tokens) of ``page`` and ``head``
  __host__ __device__ size_t record(int page, int head, int gi) const {
    const int gshift = page_shift - 4;
    return ((((size_t)page * heads + head) << gshift) + gi) * (size_t)kv_record_bytes(D);
  }
};

struct PageTableArgs {
  int R, page_shift, max_blocks, max_tokens, ring_size;
  const int32_t *cached, *added;
  int32_t *table, *ring;
  const int32_t* state;
  int32_t *seq_lens, *query_start, *slots, *positions, *state_out;
};
constexpr int kMaxTableRequests = 8192;
cudaError_t launch_page_tables(const PageTableArgs& a, int num_sms, cudaStream_t s);

cudaError_t launch_kv_append(const KvView& c, const void* k, const void* v, bool f32, long long k_stride,
                             long long v_stride, int N, const int32_t* slots, int num_sms, cudaStream_t s);
cudaError_t launch_kv_gather(const KvView& c, const int32_t* slots, int N, void* k_out, void* v_out, int num_sms,
                             cudaStream_t s);

struct KvAttnArgs;
// A request as the attention kernels take it: its rows that are written (those
// in q, at most max_q_len), its keys, and the position of its first row, which
// its true number of rows gives.
struct KvRequest {
  int qb, ql, n, first;
};

struct KvAttnArgs {
  KvView cache;
  int R, N, Hq, max_blocks, max_q_len;
  int causal, window;
  long long q_stride;
  float scale;
  const uint16_t* q;
  const int32_t *table, *seq_lens, *query_start;
  uint16_t* out;
  float* lse;
  uint8_t* workspace;
  uint32_t* status;
  int num_sms;
  WaitSettings wait;  // limit of every wait in the kernels
};
__device__ __forceinline__ KvRequest kv_request(const KvAttnArgs& a, int r) {
  KvRequest q;
  const int end = a.query_start[r + 1];
  q.qb = min(max(a.query_start[r], 0), a.N);
  q.ql = min(min(max(end, 0), a.N) - q.qb, a.max_q_len);
  q.n = (int)min((long long)max(a.seq_lens[r], 0), (long long)a.max_blocks << a.cache.page_shift);
  q.first = q.n - (max(end, q.qb) - q.qb);
  return q;
}

// Queries as f16 times a power of two a row (and kv head): the largest magnitude
// goes into [2^14, 2^15), so elements down to 2^-31 of it keep their 8 significant
// bits.  Those below lose some, the less the smaller they are: ``rest`` is the sum
// of what a row's elements lose, in units of 2^e.  A key of scale byte s moves its
// score (units of log2, factor fs = |scale| log2 e) by at most
// fs 2^e rest 6 2^(s - 127), which stays below 2^-16 for s up to kv_key_top();
// larger keys are multiplied in float32 (streaming kernel) or mark the request
// (tensor-core kernel).  An element below 2^-31 of a row's largest is rare, and its
// keys' limit lies high: queries of size 1, 128 wide: s = 146, keys of 2^19.
constexpr int kQueryExp = 14;
struct KvQueryRange {  // of some of a row's elements
  uint32_t largest = 0u, least = 0xFFFFFFFFu;  // magnitudes as bits, two at a time; ``least`` minus 1, zeros left out
  __device__ __forceinline__ void add(uint32_t w) {
    const uint32_t x = w & 0x7FFF7FFFu;
    uint32_t y;
    asm("max.u16x2 %0, %0, %1;" : "+r"(largest) : "r"(x));
    asm("add.u16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xFFFFFFFFu));
    asm("min.u16x2 %0, %0, %1;" : "+r"(least) : "r"(y));
  }
  __device__ __forceinline__ uint32_t most() const { return max(largest & 0xFFFFu, largest >> 16); }
  // does an element lose bits beside a largest of ``m`` (bits)?
  __device__ __forceinline__ bool loses(uint32_t m) const {
    const uint32_t l = min(least & 0xFFFFu, least >> 16) + 1u;
    return m < 0x7F80u && (m >> 7) > 17u + kQueryExp && l < ((m >> 7) - 17u - kQueryExp) << 7;
  }
};
// What a row that loses bits loses at least: elements below 2^-149 in units of 2^e
// are gone from its float32 differences too, 128 of them less than this.
constexpr float kQueryRest = 0x1p-120f;
// A row with an infinite or NaN element has no finite softmax over any key:
// infinite scores of one sign would pass for hidden keys, so all of its f16
// elements become NaN (and with them the scores of the keys that it sees).
__device__ __forceinline__ bool kv_query_finite(uint32_t m) { return m < 0x7F80u; }
// the row's e from its largest magnitude's bits
__device__ __forceinline__ int kv_query_exp(uint32_t m) { return m > 0u && kv_query_finite(m) ? (int)(m >> 7) - 127 - kQueryExp : 0; }
__device__ __forceinline__ int kv_exponent(float v) { return (int)((__float_as_uint(v) >> 23) & 255u) - 127; }
__device__ __forceinline__ int kv_key_top(float rest, float fs, int e) {
  // (mantissas of rest and fs below 2 each, 6 < 8: five powers of two)
  return rest > 0.f ? 127 - 16 - 5 - (kv_exponent(rest) + kv_exponent(fs) + e) : 255;
}

// First key that a row at ``pos`` sees (no sum leaves an int, whatever the window).
__device__ __forceinline__ int kv_first_key(int pos, int window) {
  return window && pos >= window ? pos - window + 1 : 0;
}

// Streaming kernels: requests of at most ``row_limit`` rows (query rows x heads
// per kv head) or marked in ``odd`` (may be null); row tiles of 8 * tiles rows
// (tiles 1 or 2).
size_t kv_stream_workspace(int D);
cudaError_t launch_kv_stream(const KvAttnArgs& a, int row_limit, const int32_t* odd, int tiles, uint8_t* ws,
                             cudaStream_t s);

// Tensor-core kernel: requests of more than ``row_limit`` rows; marks in odd [R]
// those whose scales it cannot hold, for launch_kv_stream to do over.
cudaError_t launch_kv_prompt(const KvAttnArgs& a, int row_limit, int32_t* odd, cudaStream_t s);

size_t kv_attention_workspace(const KvView& c, const kv_mxfp4_attn_t* a);
cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s);

}  // namespace moe

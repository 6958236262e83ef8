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
struct RopeArgs {
  int N, Hq, rotary_dim, max_positions, position_offset;
  long long q_stride, k_stride, v_stride;
  const void *q, *k, *v;
  const int32_t *positions, *slots;
  const float* cos_sin;
  uint16_t* q_out;
};
cudaError_t launch_kv_append_rope(const KvView& c, const RopeArgs& a, bool f32, bool pairs, int num_sms, cudaStream_t s);
cudaError_t launch_kv_gather(const KvView& c, const int32_t* slots, int N, void* k_out, void* v_out, int num_sms,
                             cudaStream_t s);

struct KvAttnArgs;
// A request as the attention kernels take it: its rows that are written (those
// in q, at most max_q_len), its keys, and the position of its first row, which
// its true number of rows gives.
struct KvRequest {
  int qb, ql, n, first;
  int causal;
  int base;  // position of its first key in its pages' table (slices of a shared prefix)
  int part;  // where its results go, for calls with a shared prefix
};

// A prefix that all requests of a call share (kv_mxfp4_attention_shared).  It is cut
// into ``splits`` slices, each a request of its own (numbers R ..) of all query rows,
// whose keys every row sees.  Results, of the requests' own keys (part 0) and of
// each slice (part 1 ..), are sums that kv_join_kernel puts together.
constexpr int kMaxSplits = 31;   // (a lane of a warp looks at each part)
constexpr int kSliceKeys = 128;  // slices start at multiples of this
struct KvShared {
  int splits = 0;  // 0: no prefix, one result a row
  int blocks = 0;  // entries of table
  int row_limit = 0;  // slices with more rows than this go to the tensor-core kernel: all, or none
  const int32_t *table = nullptr, *len = nullptr;
  float* o = nullptr;    // [part][N * Hq][D]: weighted sums of values, in units of 2^(E - 127)
  float4* ml = nullptr;  // [part][N * Hq]: reference (units of 4 log2), sum of weights, E, unused
};

// Keys of slice ``i`` of a prefix of P: the first and how many.
struct KvSlice {
  int base, n;
};
__host__ __device__ inline KvSlice kv_slice(int P, int splits, int i) {
  // (64 bits: near the top of the range a slice, rounded up, passes the largest int)
  const long long unit = (long long)splits * kSliceKeys, slice = (P + unit - 1) / unit * kSliceKeys;
  const long long base = slice * i < P ? slice * i : P;
  return {(int)base, (int)(P - base < slice ? P - base : slice)};
}

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
  KvShared sh;
};
#ifdef __CUDACC__
// Keys of the shared prefix.
__device__ __forceinline__ int kv_prefix(const KvAttnArgs& a) {
  return (int)min((long long)max(*a.sh.len, 0), (long long)a.sh.blocks << a.cache.page_shift);
}
template <bool SHARED>
__device__ __forceinline__ KvRequest kv_request(const KvAttnArgs& a, int r) {
  KvRequest q;
  q.base = 0;
  q.part = 0;
  q.causal = a.causal;
  if (SHARED && r >= a.R) {
    const KvSlice slice = kv_slice(kv_prefix(a), a.sh.splits, r - a.R);
    q.base = slice.base;
    q.part = 1 + r - a.R;
    q.causal = 0;
    q.qb = 0;
    q.ql = min(max(a.query_start[a.R], 0), a.N);
    q.n = slice.n;
    q.first = q.n;
    return q;
  }
  const int end = a.query_start[r + 1];
  q.qb = min(max(a.query_start[r], 0), a.N);
  q.ql = min(min(max(end, 0), a.N) - q.qb, a.max_q_len);
  q.n = (int)min((long long)max(a.seq_lens[r], 0), (long long)a.max_blocks << a.cache.page_shift);
  q.first = q.n - (max(end, q.qb) - q.qb);
  return q;
}
// The last request that begins at or before token ``tok``, -1 for none: 32 candidates at a time (the whole warp calls it).
__device__ __forceinline__ int kv_request_at(const KvAttnArgs& a, int tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.R;  // it is one of lo .. lo + n - 1, or the token is none's
  while (n > 1) {
    const int step = (n + 31) / 32, k = lane * step;
    const bool begun = k < n && a.query_start[lo + k] <= tok;
    const int c = __popc(__ballot_sync(0xffffffffu, begun));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  return lo;
}
// Is one of the tokens first .. last of a request that is streamed without a prefix, of at most ``limit`` rows (the whole warp
// calls it)?
__device__ __forceinline__ bool kv_few_rows_among(const KvAttnArgs& a, int G, int limit, int first, int last) {
  const int lane = threadIdx.x & 31;
  for (int r0 = max(kv_request_at(a, first), 0); r0 < a.R; r0 += 32) {
    bool few = false, past = true;
    if (r0 + lane < a.R) {
      const KvRequest q = kv_request<true>(a, r0 + lane);
      past = q.qb > last;
      few = !past && q.ql > 0 && q.qb + q.ql > first && (long long)q.ql * G <= limit;
    }
    if (__any_sync(0xffffffffu, few)) return true;
    if (__any_sync(0xffffffffu, past)) return false;
  }
  return false;
}
// Does a call with a shared prefix write the rows of token ``tok``?  Not those of an empty place of the batch, past
// max_q_len or in no request.
__device__ inline bool kv_row_counts(const KvAttnArgs& a, int tok) {
  int lo = 0, hi = a.R;  // the last request that begins at or before it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const KvRequest q = kv_request<true>(a, lo);
  return a.seq_lens[lo] >= 0 && tok >= q.qb && tok - q.qb < q.ql;
}
// Page and place in it of key ``key`` of request r.
template <bool SHARED>
__device__ __forceinline__ int kv_page(const KvAttnArgs& a, const KvRequest& q, int r, int key) {
  if (SHARED && r >= a.R) return a.sh.table[(q.base + key) >> a.cache.page_shift];
  return a.table[(size_t)r * a.max_blocks + (key >> a.cache.page_shift)];
}
template <bool SHARED>
__device__ __forceinline__ int kv_group(const KvAttnArgs& a, const KvRequest& q, int key) {
  return (((SHARED ? q.base : 0) + key) & ((1 << a.cache.page_shift) - 1)) >> 4;
}
#endif

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

// The tensor-core kernel's tiles of kKvTile keys (no sum leaves an int, whatever the keys): those that keys lo .. hi - 1 lie in,
// and whether all keys of the one from j0 on are among them.
constexpr int kKvTile = 128;
__host__ __device__ inline int kv_tiles(int lo, int hi) {
  return hi > lo ? hi / kKvTile + (hi % kKvTile != 0) - lo / kKvTile : 0;
}
__host__ __device__ inline bool kv_whole_tile(int lo, int hi, int j0) { return lo <= j0 && hi - kKvTile >= j0; }

// Streaming kernels: requests of at most ``row_limit`` rows (query rows x heads
// per kv head) or marked in ``odd`` (may be null); row tiles of 8 * tiles rows
// (tiles 1 or 2).
size_t kv_stream_workspace(int D);
cudaError_t launch_kv_stream(const KvAttnArgs& a, int row_limit, const int32_t* odd, int tiles, uint8_t* ws,
                             cudaStream_t s);

// Tensor-core kernel: requests of more than ``row_limit`` rows; marks in odd [R]
// those whose scales it cannot hold, for launch_kv_stream to do over.
cudaError_t launch_kv_prompt(const KvAttnArgs& a, int row_limit, int32_t* odd, cudaStream_t s);

// Rows of one request (query rows x heads per kv head) up to which it is streamed.
int kv_stream_rows(const KvAttnArgs& a);

// Attention with a shared prefix: how it is cut, its workspace, the call.
struct KvSharedPlan {
  int splits;   // slices of the prefix
  bool stream;  // they are streamed, else on the tensor cores
};
KvSharedPlan kv_shared_plan(const KvView& c, const kv_mxfp4_attn_t* a, int blocks);
size_t kv_shared_workspace(const KvView& c, const kv_mxfp4_attn_t* a, int splits);
cudaError_t launch_kv_shared(KvAttnArgs a, cudaStream_t s);

size_t kv_attention_workspace(const KvView& c, const kv_mxfp4_attn_t* a);
cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s);

}  // namespace moe

// Attention of a batch that shares a cached prefix (kv_mxfp4_attention_shared).
//
// With the prefix's keys j < P and a request's own keys after them, a row's softmax
// over both is joined from sums over any cut of the keys: part i has the reference
// m_i, l_i = sum 2^(s - m_i) and o_i = sum 2^(s - m_i) v, and with M = max m_i
//   out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// The prefix is read once for all rows of the batch: it is cut into slices, each a
// request of its own whose rows are all query rows of the call, which the two
// attention kernels take as they take any other request (few rows or keys:
// streamed; many: tensor cores, one CTA per 256 rows, kv head and slice).  The requests' own
// keys are parts too.  kv_join_kernel joins a row's parts.
//
// Measured, 28 / 4 heads of 128: 64 requests behind 32,768 tokens, up to 2048 own, 81 us: prefix 44
// (14 tiles of 128 keys a CTA at 2.3 us, 11 us before the first scores and after the last), own keys 20,
// items cut between CTAs 4, parts joined 6; through attention_kv_mxfp4, the prefix's pages repeated in every
// request's table, 266.  4 requests behind 100,003: 54 us (60), the streaming kernel's issue.
// Less than some 200,000 tokens of prefix times requests are not worth it (16 requests behind 10,240
// tokens 39 us either way, behind 256 32 and 19), nor are prompts, which the tensor cores
// bound (16 of 512 tokens behind 8192: 972 and 784): part sums and launches more.
#include <algorithm>

#include "kv_internal.h"

namespace moe {

namespace {

constexpr size_t kStatusBytes = 256;
// The plan is made for a GB300's SMs, so that a workspace's size depends on the sizes alone.
constexpr int kPlanSms = 152;
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// One warp a row (token x query head).  Latency-bound: the row's sums are all on their
// way while its request is looked up, kAhead parts at a time.
template <int D, int kAhead>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttnArgs a) {
  constexpr int V = D / 32;  // dims of a lane
  grid_dep_wait();
  const int lane = threadIdx.x & 31, parts = 1 + a.sh.splits;
  const long long all = (long long)a.N * a.Hq, row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= all) return;
  const float* src = a.sh.o + (size_t)row * D + V * lane;
  float v[kAhead][V];
  auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (p0 + u < parts) {
        const float* q = src + (size_t)(p0 + u) * all * D;
        if constexpr (V == 4) *reinterpret_cast<float4*>(v[u]) = __ldcs(reinterpret_cast<const float4*>(q));
        else *reinterpret_cast<float2*>(v[u]) = __ldcs(reinterpret_cast<const float2*>(q));
      }
  };
  load(0);
  // lane p: part p
  float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  if (lane < parts) ml = a.sh.ml[lane * all + row];
  const int tok = (int)(row / a.Hq), lo = kv_request_at(a, tok);
  if (lo < 0) return;
  const KvRequest q = kv_request<true>(a, lo);
  if (tok < q.qb || tok - q.qb >= q.ql) return;  // (none's, or past max_q_len)
  const bool some = ml.y != 0.f && a.seq_lens[lo] >= 0;  // (NaN too; a negative length: an empty place in the batch)
  const int E0 = some ? __float_as_int(ml.z) : -100000;
  // (a part's sums may just fit its own unit: those of up to 32 parts take 2^5 of it)
  const int E = __reduce_max_sync(0xffffffffu, E0) + 5;
  float M = some ? ml.x : -INFINITY;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float w = some ? exp2f(4.f * (ml.x - (M == -INFINITY ? 0.f : M))) : 0.f;
  float l = some ? w * ml.y : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (some) w *= exp2_int(E0 - E);  // (units of 2^0 .. 2^42: -47 at least)
  const uint32_t there = __ballot_sync(0xffffffffu, some);
  float o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = 0.f;
  for (int p0 = 0; p0 < parts; p0 += kAhead) {
    if (p0 > 0) load(p0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int p = p0 + u;
      const float wp = __shfl_sync(0xffffffffu, w, p & 31);
      if (p < parts && (there >> p & 1u)) {  // (the sums of others may be anything)
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf(v[u][k], wp, o[k]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    o[k] *= inv;
    if (l != 0.f) {  // two factors: either alone may leave the range
      const int e = min(max(E - 127, -252), 252), h = e >> 1;
      o[k] = o[k] * exp2_int(h) * exp2_int(e - h);
    }
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + V * lane);
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3]));
  else *dst = f32x2_to_bf16x2(o[0], o[1]);
  if (lane == 0 && a.lse)
    a.lse[row] = l == 0.f ? -INFINITY : M == -INFINITY ? l : fmaf(M, 2.772588722239781f, logf(l));
}

struct SharedLayout {
  size_t odd, ml, o, total;
};
SharedLayout shared_layout(int D, int R, int N, int Hq, int splits) {
  SharedLayout L;
  const size_t rows = (size_t)N * Hq * (1 + splits);
  L.odd = kStatusBytes + align256(kv_stream_workspace(D));
  L.ml = L.odd + align256(sizeof(int32_t) * ((size_t)R + splits));
  L.o = L.ml + align256(sizeof(float4) * rows);
  L.total = L.o + sizeof(float) * rows * D;
  return L;
}

}  // namespace

// How a prefix of up to ``blocks`` pages is read.  Streamed, whole, while that is thought to take
// less than the tensor cores: a row tile of 16 and kv head takes an SM 6.5 ns a key, and some 4 us for
// its pieces, which warps and CTAs share; all SMs work on it.  On the tensor cores, cut into slices: as many as
// shorten that kernel's waves (a CTA of 256 rows takes about 16 ns a key and some 5 us besides),
// against what a slice's sums cost to write and read (about 4 bytes a picosecond); 9 us for
// the launch and its marks.  The constants are of 128-wide heads; a fit to times of both gives 6.9 ns
// and 3.6 us, 18 ns and 2 us, and 7 us for the launch, beside what both ways share; what counts is the
// choice.  Measured with both ways and up to nine cuts each, 351 batches (1 to 256 requests, 16 to 100,352
// keys, 1 to 8 kv heads of 1 to 16 query heads, 64 and 128 wide): it takes 0.1 % more than the best of them on average,
// 8 % at most.  Streamed and on the tensor cores, 4 x 7 heads of 128, caches cold: 64 requests 16 keys 24 and 43
// us, 2560 41 and 44, 5120 55 and 47; 16 requests 10,240 keys 39 and 45, 30,720 68 and 56; 128 requests 256 keys
// 35 and 41; 28 rows, 100,352 keys 67 and 97.
KvSharedPlan kv_shared_plan(const KvView& c, const kv_mxfp4_attn_t* a, int blocks) {
  const long long rows = (long long)a->N * (a->Hq / c.heads);
  const long long tiles = (rows + 255) / 256 * c.heads, keys = (long long)blocks << c.page_shift;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxSplits; ++s) {
    const long long slice = (keys + (long long)s * kSliceKeys - 1) / ((long long)s * kSliceKeys) * kSliceKeys;
    const double t = (double)((tiles * s + kPlanSms - 1) / kPlanSms) * (16e-9 * slice + 5e-6) +
                     (double)s * a->N * a->Hq * c.D * 8 / 4e12;
    if (s == 1 || t < least) {
      least = t;
      best = s;
    }
  }
  const double items = (double)((rows + 15) / 16 * c.heads);
  const double streamed = items * (6.5e-9 * keys + 4e-6 * std::min(keys, 256LL) / 256) / kPlanSms + 3e-6;
  if (streamed <= least + 9e-6) return {1, true};
  return {best, false};
}

size_t kv_shared_workspace(const KvView& c, const kv_mxfp4_attn_t* a, int splits) {
  return shared_layout(c.D, a->R, a->N, a->Hq, splits).total;
}

cudaError_t launch_kv_shared(KvAttnArgs a, cudaStream_t s) {
  const int G = a.Hq / a.cache.heads;
  const SharedLayout L = shared_layout(a.cache.D, a.R, a.N, a.Hq, a.sh.splits);
  a.sh.ml = reinterpret_cast<float4*>(a.workspace + L.ml);
  a.sh.o = reinterpret_cast<float*>(a.workspace + L.o);
  uint8_t* ws = a.workspace + kStatusBytes;
  const long long all = (long long)a.N * G, own = (long long)a.max_q_len * G;
  const int limit = kv_stream_rows(a);
  int32_t* odd = nullptr;
  cudaError_t e;
  const bool stream = a.sh.row_limit > 0;
  if (!stream || own > limit) {
    odd = reinterpret_cast<int32_t*>(a.workspace + L.odd);
    if ((e = launch_kv_prompt(a, limit, odd, s)) != cudaSuccess) return e;
  }
  // row tiles of 8 where the streamed rows fit (as without a prefix); a streamed prefix with more rows
  // takes tiles of 16, unless the requests' own keys, thought to be half of their tables', weigh more: a
  // tile of 8 takes 4.6 ns a key, one of 16 6.5
  long long streamed = own <= limit ? own : G;
  if (stream && all > 8) {
    if (0.7 * a.max_blocks / 2 * a.R < (double)((all + 15) / 16) * a.sh.blocks) streamed = all;
  }
  if ((e = launch_kv_stream(a, limit, odd, streamed <= 8 ? 1 : 2, ws, s)) != cudaSuccess) return e;
  const dim3 grid((unsigned)(((long long)a.N * a.Hq + 7) / 8));
  // (8 parts at a time leave room for twice the rows on an SM: 256 requests of 6 parts 86 us
  // in all, 89 with 16 at a time; 64 of 20 parts 76, with 8 79)
  const bool few = 1 + a.sh.splits <= 8;
  auto kern = a.cache.D == 128 ? (few ? kv_join_kernel<128, 8> : kv_join_kernel<128, 16>)
                               : (few ? kv_join_kernel<64, 8> : kv_join_kernel<64, 16>);
  return launch_kernel(kern, grid, dim3(256), 0, s, true, false, a);
}

}  // namespace moe

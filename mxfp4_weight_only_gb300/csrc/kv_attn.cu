// Attention over the 4-bit KV cache (kv_mxfp4_attention).
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(S_j - max S), S_j = scale q . k_j
// over a row's visible keys, in one pass with a running maximum and sum.
#include "common.cuh"
#include "kv_internal.h"

namespace moe {

namespace {

// One warp per query row: 32 keys at a time, a lane per key for the scores, a
// lane per 2 (or 4) dimensions for the weighted sum.
template <int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(const KvAttnArgs a) {
  constexpr int NB = D / 32, E = D / 32;  // scale blocks of a row; dimensions of a lane
  __shared__ float qs[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + warp;
  if (row >= (long long)a.N * a.Hq) return;
  const int tok = (int)(row / a.Hq), h = (int)(row - (long long)tok * a.Hq);
  // the request of this token: the last one that starts at or before it
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const int r = lo, qb = a.query_start[r], ql = a.query_start[r + 1] - qb;
  const int i = tok - qb;
  if (i < 0 || i >= ql || i >= a.max_q_len) return;
  const KvView& c = a.cache;
  const int page = 1 << c.page_shift;
  const int n = (int)min((long long)max(a.seq_lens[r], 0), (long long)a.max_blocks * page);
  const int pos = n - ql + i;
  const int end = a.causal ? min(n, pos + 1) : n;
  const int begin = a.window ? max(0, pos - a.window + 1) : 0;
  const int kvh = h / (a.Hq / c.heads);
  const uint16_t* q = a.q + (size_t)tok * a.q_stride + (size_t)h * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf16_lo(q[d]) * a.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int j0 = begin; j0 < end; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < end) {
      const int pg = a.table[(size_t)r * a.max_blocks + (j >> c.page_shift)];
      if (pg >= 0 && pg < c.num_pages) {
        const int off = j & (page - 1), t = off & 15;
        const uint8_t* rec = c.data + c.record(pg, kvh, off >> 4);
        s = 0.f;
        for (int b = 0; b < NB; ++b) {
          const uint32_t sb = rec[16 * D + t * NB + b], sv = rec[16 * D + D / 2 + t * NB + b];
          float acc = 0.f;
          for (int w = 0; w < 4; ++w) {
            const uint32_t codes = *reinterpret_cast<const uint32_t*>(rec + ((t * 4 + w) * NB + b) * 4);
            uint32_t x[4];
            e2m1x8_to_f16x8(codes, x[0], x[1], x[2], x[3]);
            const float* qq = qs[warp] + 32 * b + 8 * w;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc += qq[2 * e] * f16_lo(x[e]) + qq[2 * e + 1] * f16_hi(x[e]);
          }
          s += acc * e8m0_to_float(sb);
          if (sb == 255u || sv == 255u) s = __uint_as_float(0x7FC00000u);
        }
      }
    }
    float mx = s;
    bool nan = s != s;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    nan = __any_sync(0xffffffffu, nan);
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY && !nan) continue;
    const float base = mn == -INFINITY ? 0.f : mn;
    const float al = __expf(m - base);
    const float p = __expf(s - base);
    l *= al;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= al;
    m = mn;
    for (int k = 0; k < 32 && j0 + k < end; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      l += pk;
      if (pk == 0.f) continue;  // hidden keys, and those whose weight rounds to nothing
      const int jj = j0 + k;
      const int pg = a.table[(size_t)r * a.max_blocks + (jj >> c.page_shift)];
      const int off = jj & (page - 1), t = off & 15;
      const uint8_t* rec = c.data + c.record(pg, kvh, off >> 4);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = 32 * e + lane, by = d >> 1;
        const int at = 8 * D + ((((((t >> 3) * 8 + ((by >> 1) & 7)) * 4 + ((t >> 1) & 3)) * 2 + (t & 1)) * NB) + e) * 2 + (by & 1);
        const uint32_t code = (rec[at] >> (4 * (d & 1))) & 15u;
        uint32_t x[4];
        e2m1x8_to_f16x8(code, x[0], x[1], x[2], x[3]);
        o[e] += pk * 0x1p-12f * (f16_lo(x[0]) * e8m0_to_float(rec[16 * D + D / 2 + t * NB + e]));
      }
    }
  }
  // (the sum is kept 2^12 times smaller, so that it stays finite before the division)
  const float inv = l == 0.f ? 0.f : 0x1p12f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[(size_t)row * D + 32 * e + lane] = f32_to_bf16_bits(o[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m + __logf(l);
}

}  // namespace

size_t kv_attention_workspace(const KvView&, const kv_mxfp4_attn_t*) { return 256; }

cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.N * a.Hq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (a.cache.D == 128) attn_rows_kernel<128><<<grid, 128, 0, s>>>(a);
  else attn_rows_kernel<64><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe

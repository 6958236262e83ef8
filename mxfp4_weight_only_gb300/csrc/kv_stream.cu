// Attention over the 4-bit KV cache, few query rows per request: the cache is
// streamed once, HBM-bound (kv_mxfp4_attention, decode and short drafts).
//
// One pass with a running maximum and sum per query row.  A warp takes 16-token
// records of one (request, kv head, row tile of 8 NT rows) one after another:
//   S^T[16 tokens][rows] = K Q^T      m16n8k16 MMAs, f16, per 32-value block,
//                                     times the block's 2^(s-127) in float32
//   p = 2^(S f - m)                   f: scale, log2 e, the row's exponent
//   O^T[dims][rows] += V^T (p 2^(sv)) m16n8k16 MMAs, bf16; the value scale is
//                                     folded into the weights, per 32 dims
// The record is laid out so that every lane finds its operands of these MMAs in
// two 16-byte words of keys and two of values (conflict-free shared loads, no
// shuffles).  Queries enter as f16 scaled by a power of two per row (exact: 8
// significant bits), keys as f16 (exact).  Weights enter as the sum of two bf16
// (16 bits, two MMAs: the tensor pipe has room), which keeps a weight of any
// size where the heavier keys' values are zero (one f16 weight, 11 bits, loses
// those below 2^-32; one bf16 weight has 8 bits).  Value scales outside
// 2^-63 .. 2^64 (or NaN bytes) take an exact float32 path (add_group_f32).
//
// Work: a unit is one record of one item (request, kv head, row tile); the
// units of all items in order are cut into equal runs, one per warp of a
// one-CTA-per-SM grid, so ragged batches balance without a host-side plan: every
// CTA finds its place by a prefix sum over the requests.  Each warp streams its
// run through a private ring of bulk copies (one per record) without any
// barrier with other warps.  Items cut between warps are merged in shared
// memory, items cut between CTAs through the workspace by kv_merge_kernel.
#include "common.cuh"
#include "kv_internal.h"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kKvWaitNs = kWaitLimitNs;

template <int D, int NT>
struct StreamCfg {
  static constexpr int NB = D / 32;
  static constexpr int kWarps = NT == 1 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRec = 17 * D;
  static constexpr int kStages = (NT == 1 ? 4 : 8) * (128 / D);
  static constexpr int kCols = 8 * NT;
  // a piece in shared memory: O [kCols][D + 4] float, m, l [kCols], reference scale E
  static constexpr int kPieceFloats = kCols * (D + 4) + 2 * kCols + 4;
  static constexpr int kRingBytes = kStages * kRec;
  static constexpr int kStash = kPieceFloats * 4;
  static_assert(kStash <= kRingBytes, "a warp's last piece is stored in its drained ring");
  static constexpr int kSmem = kWarps * (kRingBytes + kStash);
};

// Workspace after the status region: per CTA two part headers and two parts.
struct PartHead {
  long long item;  // first unit of the item
  int units;       // its units
  int r, pair;     // request; kv head * row tiles + row tile
  int starts;      // 1: the item starts in this CTA and ends in a later one
  int E;
  int pad;
};

__host__ __device__ constexpr size_t part_floats(int cols, int D) { return (size_t)cols * D + 2 * cols; }

struct StreamParams {
  KvAttnArgs a;
  int G;           // query heads per kv head
  int row_limit;   // requests with more rows than this are not this kernel's
  int max_ctas;
  PartHead* heads;   // [grid][2]
  float* parts;      // [grid][2][part_floats]
  long long* plan;   // [2]: units, active warps
};

// What a request asks for: rows, the record range any of its rows can see.
struct Req {
  int qb, ql, n, glo, ng, rt;
  __device__ __forceinline__ long long units(int heads) const { return (long long)ng * heads * rt; }
};

template <int COLS>
__device__ __forceinline__ Req request(const StreamParams& p, int r) {
  const KvAttnArgs& a = p.a;
  Req q;
  q.qb = min(max(a.query_start[r], 0), a.N);
  q.ql = min(min(max(a.query_start[r + 1], 0), a.N) - q.qb, a.max_q_len);
  const long long cap = (long long)a.max_blocks << a.cache.page_shift;
  const int full = a.seq_lens[r];
  q.n = (int)min((long long)max(full, 0), cap);
  const long long rows = (long long)max(q.ql, 0) * p.G;
  const bool mine = rows > 0 && rows <= p.row_limit;
  q.rt = mine ? (int)((rows + COLS - 1) / COLS) : 0;
  q.glo = a.window ? max(0, q.n - q.ql - a.window + 1) >> 4 : 0;
  q.ng = mine ? ((q.n + 15) >> 4) - q.glo : 0;
  return q;
}

__device__ __forceinline__ uint32_t movm(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t bf16mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// D += A * B for one m16n8k16 tile, bf16 inputs, f32 accumulate.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 codes of each of two tokens (4 dims of two blocks) -> per block and
// dim the bf16 pair (token a low, token b high), exact: codes to f16 pairs of
// two dims, each value to float32 (fused multiply-add pipe), whose high halves
// are the bf16 values, put together by a byte permute.
__device__ __forceinline__ void token_pairs(uint32_t ta, uint32_t tb, uint32_t (&blk0)[4], uint32_t (&blk1)[4]) {
  uint32_t x[4], y[4];
  e2m1x8_to_f16x8(ta, x[0], x[1], x[2], x[3]);
  e2m1x8_to_f16x8(tb, y[0], y[1], y[2], y[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = prmt(__float_as_uint(f16_lo(x[i])), __float_as_uint(f16_lo(y[i])), 0x7632u);
    const uint32_t hi = prmt(__float_as_uint(f16_hi(x[i])), __float_as_uint(f16_hi(y[i])), 0x7632u);
    if (i < 2) {
      blk0[2 * i] = lo;
      blk0[2 * i + 1] = hi;
    } else {
      blk1[2 * (i - 2)] = lo;
      blk1[2 * (i - 2) + 1] = hi;
    }
  }
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float lg2(float v) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 2^e for any e: two factors, so that results below the normal range and up to 2^254 apart work out.
__device__ __forceinline__ float mul_pow2(float v, int e) {
  const int c = min(max(e, -252), 252), h = c >> 1;
  return v * exp2_int(h) * exp2_int(c - h);
}

// The lane's words of 16 tokens of keys (or values): NB words per half.
template <int NB>
__device__ __forceinline__ void load_words(const uint8_t* p, int lane, uint32_t (&w)[2][NB]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (NB == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + (h * 32 + lane) * 16);
      w[h][0] = u.x;
      w[h][1] = u.y;
      w[h][NB - 2] = u.z;
      w[h][NB - 1] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p + (h * 32 + lane) * 8);
      w[h][0] = u.x;
      w[h][1] = u.y;
    }
  }
}

// A token's NB scale bytes in the low bytes of a word; unused bytes hold ``fill``'s.
template <int NB>
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p, int tok, uint32_t fill) {
  if (NB == 4) return *reinterpret_cast<const uint32_t*>(p + 4 * tok);
  return *reinterpret_cast<const uint16_t*>(p + 2 * tok) | (fill & 0xFFFF0000u);
}

// One item's state in a warp.  Lane (g, t) = (lane / 4, lane % 4) holds, for its
// two rows 2t, 2t+1 of each row tile of 8, dims 4g .. 4g+3 of every block.
template <int D, int NT>
struct Acc {
  static constexpr int NB = D / 32;
  float o[NT][NB][2][4];  // [tile][block][dims 01 / 23][dim a rows 2t, 2t+1; dim b rows 2t, 2t+1]
  float m[NT][2], l[NT][2];
  int E;
};

// O += p V in float32 for one record, any value scales (the exceptional case):
// the weights of token k come from the lane that holds them.  O is kept in units
// of 2^(E - 127).
template <int D, int NT>
__device__ __noinline__ void add_group_f32(Acc<D, NT>& A, const uint8_t* rec, int lane, const float (&p)[NT][4],
                                           int valid) {
  constexpr int NB = D / 32;
  const int g = lane >> 2, t = lane & 3;
  for (int k = 0; k < 16; ++k) {
    const int src = (k & 7) * 4 + t;
    float w[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      w[i][0] = __shfl_sync(0xffffffffu, k < 8 ? p[i][0] : p[i][2], src);
      w[i][1] = __shfl_sync(0xffffffffu, k < 8 ? p[i][1] : p[i][3], src);
    }
    if (k >= valid) continue;
    const uint8_t* vc = rec + 8 * D + ((((k >> 3) * 8 + g) * 4 + ((k >> 1) & 3)) * 2 + (k & 1)) * NB * 2;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t s = rec[16 * D + D / 2 + k * NB + b];
      if (s == 255u) continue;  // the token's weights are NaN where it is seen
      uint32_t x[4];
      e2m1x8_to_f16x8(*reinterpret_cast<const uint16_t*>(vc + 2 * b), x[0], x[1], x[2], x[3]);
      const float v[4] = {f16_lo(x[0]), f16_hi(x[0]), f16_lo(x[1]), f16_hi(x[1])};
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            A.o[i][b][d >> 1][(d & 1) * 2 + c] += mul_pow2(w[i][c] * v[d], (int)s - A.E);
    }
  }
}

// Largest value-scale byte (255 excluded) of the valid tokens of a record, warp-wide.
template <int NB>
__device__ __forceinline__ int largest_scale(uint32_t w0, uint32_t w1, bool ok0, bool ok1) {
  int mx = 0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int x = (w0 >> (8 * b)) & 255, y = (w1 >> (8 * b)) & 255;
    if (ok0 && x != 255) mx = max(mx, x);
    if (ok1 && y != 255) mx = max(mx, y);
  }
  return __reduce_max_sync(0xffffffffu, mx);
}

// Any of a word's first NB bytes outside 64 .. 191 and not 0?
template <int NB>
__device__ __forceinline__ bool unusual_scale(uint32_t w) {
  bool r = false;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t x = (w >> (8 * b)) & 255u;
    r |= x != 0u && x - 64u > 127u;
  }
  return r;
}

// Any byte of a word equal to 255?
__device__ __forceinline__ bool has_nan_byte(uint32_t w, int nb) {
  bool r = false;
  for (int b = 0; b < nb; ++b) r |= ((w >> (8 * b)) & 255u) == 255u;
  return r;
}

template <int D, int NT>
__global__ void __launch_bounds__(StreamCfg<D, NT>::kThreads, 1) kv_stream_kernel(const StreamParams p) {
  using C = StreamCfg<D, NT>;
  constexpr int NB = C::NB, W = C::kWarps, S = C::kStages, REC = C::kRec, COLS = C::kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W * S];
  __shared__ long long sc_scan[W], start_off[W];
  __shared__ int start_r[W];
  __shared__ PartHead ph[W][2];    // pieces left by each warp: [0] its first, [1] its last
  __shared__ int empties[C::kThreads], n_empty;
  const KvAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRingBytes;
  float* stash = reinterpret_cast<float*>(smem + W * C::kRingBytes + warp * C::kStash);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&bars[warp * S + s], 1);
    fence_barrier_init();
    ph[warp][0].units = ph[warp][1].units = 0;
    start_r[warp] = -1;
  }
  grid_dep_launch_dependents();

  // ---------------------------------------------------------------- units of all requests
  const int H = a.cache.heads;
  long long total = 0;
  const int chunks = (a.R + C::kThreads - 1) / C::kThreads;
  long long my_first = 0;  // first unit of request tid (first chunk), kept for the search below
  for (int ch = 0; ch < chunks; ++ch) {
    const int r = ch * C::kThreads + tid;
    long long u = 0;
    if (tid == 0) n_empty = 0;
    __syncthreads();
    if (r < a.R) {
      const Req q = request<COLS>(p, r);
      u = q.units(H);
      // requests without a key: their rows are zeros, written by one CTA each
      if (u == 0 && q.rt > 0 && r % gridDim.x == blockIdx.x) empties[atomicAdd(&n_empty, 1)] = r;
    }
    long long incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sc_scan[warp] = incl;
    __syncthreads();
    long long before = total, sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += sc_scan[w];
      sum += sc_scan[w];
    }
    my_first = before + incl - u;
    total += sum;
    for (int k = 0; k < n_empty; ++k) {
      const Req q = request<COLS>(p, empties[k]);
      const long long rows = (long long)q.ql * a.Hq;
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)q.qb * a.Hq * D);
      for (long long i = tid; i < rows * (D / 8); i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (long long i = tid; i < rows; i += C::kThreads) a.lse[(size_t)q.qb * a.Hq + i] = -INFINITY;
    }
    __syncthreads();
  }
  const long long U = total;
  const long long all_warps = (long long)gridDim.x * W;
  const long long A_w = max(min(all_warps, U), 1ll);  // active warps
  auto begin_of = [&](long long w) { return w >= A_w ? U : w * U / A_w; };
  const long long gw0 = (long long)blockIdx.x * W, cta_lo = begin_of(gw0), cta_hi = begin_of(gw0 + W);
  if (blockIdx.x == 0 && tid == 0) {
    p.plan[0] = U;
    p.plan[1] = A_w;
  }
  if (tid < 2) p.heads[2 * blockIdx.x + tid].units = 0;
  if (cta_lo >= cta_hi) return;
  // the request in which each warp's run starts: the thread that holds it tells
  long long base = 0;
  for (int ch = 0; ch < chunks; ++ch) {
    const int r = ch * C::kThreads + tid;
    long long u = 0, first;
    if (r < a.R) u = request<COLS>(p, r).units(H);
    if (chunks == 1) {
      first = my_first;
    } else {
      long long incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sc_scan[warp] = incl;
      __syncthreads();
      first = base + incl - u;
      long long sum = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w < warp) first += sc_scan[w];
        sum += sc_scan[w];
      }
      base += sum;
    }
    if (u > 0 && first < cta_hi && first + u > cta_lo) {
      for (int w = 0; w < W; ++w) {
        const long long b = begin_of(gw0 + w);
        if (b >= first && b < first + u && b < begin_of(gw0 + w + 1)) {
          start_r[w] = r;
          start_off[w] = b - first;
        }
      }
    }
    __syncthreads();
  }

  // ---------------------------------------------------------------- this warp's run
  const long long u_lo = begin_of(gw0 + warp), u_hi = begin_of(gw0 + warp + 1);
  const int n_units = (int)(u_hi - u_lo);
  if (n_units > 0) {
    // record addresses, 32 units at a time, one per lane; null for a page outside the cache
    int br = start_r[warp];
    long long bo = start_off[warp];
    auto addresses = [&](int i0) -> const uint8_t* {
      const uint8_t* ptr = nullptr;
      int r = br;
      long long off = bo + lane;
      if (i0 + lane < n_units) {
        Req q = request<COLS>(p, r);
        while (off >= q.units(H)) {
          off -= q.units(H);
          q = request<COLS>(p, ++r);
        }
        const int pair = (int)(off / q.ng), gi = q.glo + (int)(off - (long long)pair * q.ng);
        const int tok = gi << 4;
        const int pg = a.table[(size_t)r * a.max_blocks + (tok >> a.cache.page_shift)];
        if (pg >= 0 && pg < a.cache.num_pages)
          ptr = a.cache.data + a.cache.record(pg, pair / q.rt, (tok & ((1 << a.cache.page_shift) - 1)) >> 4);
      }
      // the next 32 start after lane 31's
      br = __shfl_sync(0xffffffffu, r, 31);
      bo = __shfl_sync(0xffffffffu, off, 31) + 1;
      return ptr;
    };
    const uint64_t policy = l2_policy_evict_first();
    const uint8_t* cur = addresses(0);
    const uint8_t* nxt = n_units > 32 ? addresses(32) : nullptr;
    uint64_t* bar = bars + warp * S;
    auto issue = [&](int i, const uint8_t* c0, const uint8_t* c1, int batch) {
      // unit i lies in batch ``batch`` (addresses c0) or the next one (c1)
      const unsigned long long v = (unsigned long long)((i >> 5) == batch ? c0 : c1);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, v, i & 31));
      if (lane == 0) {
        const int s = i % S;
        if (src) {
          mbar_arrive_expect_tx(&bar[s], REC);
          bulk_g2s(ring + s * REC, src, REC, &bar[s], policy);
        } else {
          mbar_arrive(&bar[s]);
        }
      }
    };
    for (int i = 0; i < min(S, n_units); ++i) issue(i, cur, nxt, 0);

    int cr = start_r[warp];
    long long co = start_off[warp];
    bool alive = true;
    int i = 0;
    while (i < n_units && alive) {
      // ------------------------------------------------------------ next item
      Req q = request<COLS>(p, cr);
      while (co >= q.units(H)) {
        co -= q.units(H);
        q = request<COLS>(p, ++cr);
      }
      const int pair = (int)(co / q.ng), g0 = (int)(co - (long long)pair * q.ng);
      const int kvh = pair / q.rt, rt = pair - kvh * q.rt;
      const int len = min(q.ng - g0, n_units - i);
      const long long item = u_lo + i - g0;
      // queries: f16 times a power of two per row; f folds scale and log2 e
      uint32_t qf[NT][NB][4];
      float f[NT][2];
      int lo[NT][2], hi[NT][2];
      int shift = 0;
      {
        const int rows = q.ql * p.G;
        float fcol[NT];
        int fe = -10000;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = rt * COLS + nt * 8 + g;
          float mx = 0.f;
          uint4 u[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) u[b] = make_uint4(0, 0, 0, 0);
          if (c < rows) {
            const int row = c / p.G, hq = c - row * p.G;
            const uint16_t* qp = a.q + (size_t)(q.qb + row) * a.q_stride + (size_t)(kvh * p.G + hq) * D + 8 * t;
#pragma unroll
            for (int b = 0; b < NB; ++b) u[b] = __ldg(reinterpret_cast<const uint4*>(qp + 32 * b));
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t w[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // largest magnitude into [8, 16)
          const int e = mx > 0.f && mx < INFINITY ? (int)(__float_as_uint(mx) >> 23) - 127 - 3 : 0;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t w[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              qf[nt][b][k] = f32x2_to_f16x2(mul_pow2(bf16_lo(w[k]), -e), mul_pow2(bf16_hi(w[k]), -e));
          }
          fcol[nt] = mul_pow2(a.scale * kLog2e, e);
          if (c < rows && fcol[nt] != 0.f) fe = max(fe, (int)((__float_as_uint(fcol[nt]) >> 23) & 255u) - 127);
        }
        // factors of an unusual size go into the key scales, so that partial sums
        // stay near the scores' size
        fe = __reduce_max_sync(0xffffffffu, fe);
        shift = fe > -9999 && (fe > 40 || fe < -40) ? min(max(fe, -126), 126) : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float v = mul_pow2(fcol[nt], -shift);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            f[nt][k] = __shfl_sync(0xffffffffu, v, 4 * (2 * t + k));
            const int c = rt * COLS + nt * 8 + 2 * t + k;
            const int row = c / p.G;
            const int pos = q.n - q.ql + row;
            const bool real = c < rows;
            hi[nt][k] = real && a.causal ? min(q.n, pos + 1) : q.n;
            lo[nt][k] = real && a.window ? max(0, pos - a.window + 1) : 0;
          }
        }
      }
      int lo_max = 0, hi_min = q.n;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          lo_max = max(lo_max, lo[nt][k]);
          hi_min = min(hi_min, hi[nt][k]);
        }
      lo_max = __reduce_max_sync(0xffffffffu, lo_max);
      hi_min = __reduce_min_sync(0xffffffffu, hi_min);

      Acc<D, NT> A;
      A.E = 127;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < 8; ++k) A.o[nt][b][k >> 2][k & 3] = 0.f;
        A.m[nt][0] = A.m[nt][1] = -INFINITY;
        A.l[nt][0] = A.l[nt][1] = 0.f;
      }

      for (int k = 0; k < len; ++k, ++i) {
        const int s = i % S;
        if (!mbar_wait(&bar[s], (i / S) & 1, a.status, kKvWaitNs)) {
          alive = false;
          break;
        }
        const uint8_t* rec = ring + s * REC;
        const bool present = __shfl_sync(0xffffffffu, (unsigned long long)cur, i & 31) != 0ull;
        if (present) {
          const int j0 = (q.glo + g0 + k) << 4;
          const int valid = q.n - j0;  // tokens of the record that exist (above 16: all)
          // ---------------------------------------------------- scores
          float sc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
          uint32_t kw[2][NB];
          load_words<NB>(rec, lane, kw);
          uint32_t ks0 = scale_word<NB>(rec + 16 * D, g, 0x7F7F7F7Fu), ks1 = scale_word<NB>(rec + 16 * D, g + 8, 0x7F7F7F7Fu);
          uint32_t vs0 = scale_word<NB>(rec + 16 * D + D / 2, g, 0x7F7F7F7Fu),
                   vs1 = scale_word<NB>(rec + 16 * D + D / 2, g + 8, 0x7F7F7F7Fu);
          if (valid < 16) {
            if (g >= valid) ks0 = 0x7F7F7F7Fu;
            if (g + 8 >= valid) ks1 = 0x7F7F7F7Fu;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t x[4], y[4];
            e2m1x8_to_f16x8(kw[0][b], x[0], x[1], x[2], x[3]);
            e2m1x8_to_f16x8(kw[1][b], y[0], y[1], y[2], y[3]);
            float s0, s1;
            if (shift == 0) {
              // byte -> 2^(s-127): 0 gives 0 (for 2^-127), 255 infinity, which poisons the score below
              s0 = __uint_as_float((b < 3 ? ks0 << (23 - 8 * b) : ks0 >> 1) & 0x7F800000u);
              s1 = __uint_as_float((b < 3 ? ks1 << (23 - 8 * b) : ks1 >> 1) & 0x7F800000u);
            } else {
              const int b0 = (ks0 >> (8 * b)) & 255, b1 = (ks1 >> (8 * b)) & 255;
              s0 = __uint_as_float((uint32_t)(b0 == 255 ? 255 : min(max(b0 + shift, 0), 254)) << 23);
              s1 = __uint_as_float((uint32_t)(b1 == 255 ? 255 : min(max(b1 + shift, 0), 254)) << 23);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4];
              const float z[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16_16816(d, x[0], y[0], x[1], y[1], qf[nt][b][0], qf[nt][b][1], z);
              mma_f16_16816(d, x[2], y[2], x[3], y[3], qf[nt][b][2], qf[nt][b][3], d);
              sc[nt][0] = fmaf(d[0], s0, sc[nt][0]);
              sc[nt][1] = fmaf(d[1], s0, sc[nt][1]);
              sc[nt][2] = fmaf(d[2], s1, sc[nt][2]);
              sc[nt][3] = fmaf(d[3], s1, sc[nt][3]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float v = sc[nt][c] * f[nt][c & 1];
              sc[nt][c] = fmaf(v, 0.f, v);  // infinities become NaN
            }
          // ---------------------------------------------------- value scales
          if (valid < 16) {
            if (g >= valid) vs0 = 0x7F7F7F7Fu;
            if (g + 8 >= valid) vs1 = 0x7F7F7F7Fu;
          }
          // the common case: every byte in 64 .. 191 (its two top bits differ) and O in units of 1
          bool wide = A.E != 127;
          if (__any_sync(0xffffffffu, ((vs0 ^ (vs0 << 1)) & (vs1 ^ (vs1 << 1)) & 0x80808080u) != 0x80808080u) || wide) {
            // zero bytes are as good: blocks below 2^-124, multiplied by 0
            wide |= (bool)__any_sync(0xffffffffu, unusual_scale<NB>(vs0) || unusual_scale<NB>(vs1));
            if (wide) {
              const int mx = largest_scale<NB>(vs0, vs1, g < valid, g + 8 < valid);
              if (mx > A.E + 60) {  // sums of values this large would overflow in the present unit
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int c = 0; c < 8; ++c) A.o[nt][b][c >> 2][c & 3] = mul_pow2(A.o[nt][b][c >> 2][c & 3], A.E - mx);
                A.E = mx;
              }
              // a NaN value block makes its token NaN
              const float nan = __uint_as_float(0x7FC00000u);
              const bool n0 = has_nan_byte(vs0, NB), n1 = has_nan_byte(vs1, NB);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (n0) sc[nt][0] = sc[nt][1] = nan;
                if (n1) sc[nt][2] = sc[nt][3] = nan;
              }
            }
          }
          // ---------------------------------------------------- masks
          if (j0 + 16 > hi_min || j0 < lo_max) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int j = j0 + g + (c >> 1) * 8;
                if (j >= hi[nt][c & 1] || j < lo[nt][c & 1]) sc[nt][c] = -INFINITY;
              }
          }
          // ---------------------------------------------------- running maximum and sum
          float mn[NT][2];
          bool grow = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = fmaxf(sc[nt][c], sc[nt][c + 2]);
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              mn[nt][c] = fmaxf(A.m[nt][c], v);
              grow |= mn[nt][c] > A.m[nt][c];
            }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float al[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                al[c] = mn[nt][c] == -INFINITY ? 1.f : ex2(A.m[nt][c] - mn[nt][c]);
                A.l[nt][c] *= al[c];
                A.m[nt][c] = mn[nt][c];
              }
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 8; ++c) A.o[nt][b][c >> 2][c & 3] *= al[c & 1];
            }
          }
          uint32_t pk[NT][2][2];  // [token g / g + 8][upper 8 bits / the rest]
          float pw[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float m0 = A.m[nt][c & 1];
              // (a row that has seen nothing yet keeps weight 0)
              pw[nt][c] = ex2(sc[nt][c] - (m0 == -INFINITY ? 0.f : m0));
              A.l[nt][c & 1] += pw[nt][c];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u = __float_as_uint(pw[nt][2 * h]), v = __float_as_uint(pw[nt][2 * h + 1]);
              pk[nt][h][0] = prmt(u, v, 0x7632u);
              pk[nt][h][1] = f32x2_to_bf16x2(pw[nt][2 * h] - __uint_as_float(u & 0xFFFF0000u),
                                             pw[nt][2 * h + 1] - __uint_as_float(v & 0xFFFF0000u));
            }
          }
          // ---------------------------------------------------- weighted sum
          if (!wide) {
            uint32_t vw[2][NB];
            load_words<NB>(rec + 8 * D, lane, vw);
#pragma unroll
            for (int bp = 0; bp < NB / 2; ++bp) {
              // [half][block of the pair][dim]: two tokens, one dimension
              uint32_t xv[2][2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) token_pairs(vw[h][bp], vw[h][NB / 2 + bp], xv[h][0], xv[h][1]);
#pragma unroll
              for (int bb = 0; bb < 2; ++bb) {
                const int b = 2 * bp + bb;
                // 2^(s-127) as bf16, twice in a word
                const uint32_t sel = 0x0404u | ((uint32_t)b << 4) | ((uint32_t)b << 12);
                const uint32_t e0 = prmt(vs0, 0u, sel) >> 1, e1 = prmt(vs1, 0u, sel) >> 1;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int w = 0; w < 2; ++w) {
                    const uint32_t p0 = movm(bf16mul2(pk[nt][0][w], e0)), p1 = movm(bf16mul2(pk[nt][1][w], e1));
                    mma_bf16_16816(A.o[nt][b][0], xv[0][bb][0], xv[0][bb][1], xv[1][bb][0], xv[1][bb][1], p0, p1);
                    mma_bf16_16816(A.o[nt][b][1], xv[0][bb][2], xv[0][bb][3], xv[1][bb][2], xv[1][bb][3], p0, p1);
                  }
              }
            }
          } else {
            // (copies, so that the common path keeps both in registers)
            Acc<D, NT> B = A;
            float w[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) w[nt][c] = pw[nt][c];
            add_group_f32<D, NT>(B, rec, lane, w, valid);
            A = B;
          }
        }
        // the stage is free: the record S units on
        __syncwarp();
        if (i + S < n_units) issue(i + S, cur, nxt, i >> 5);
        if ((i & 31) == 31) {
          cur = nxt;
          nxt = i + 33 < n_units ? addresses(i + 33) : nullptr;
        }
      }
      co += len;
      // ------------------------------------------------------------ the item, or a piece of it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float l = A.l[nt][c];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          A.l[nt][c] = l;
        }
      if (g0 == 0 && len == q.ng) {
        const int rows = q.ql * p.G;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = rt * COLS + nt * 8 + 2 * t + c;
            if (col < rows) {
              const int row = col / p.G, hq = kvh * p.G + col - row * p.G;
              const size_t at = (size_t)(q.qb + row) * a.Hq + hq;
              const float l = A.l[nt][c], inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                float v[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = mul_pow2(A.o[nt][b][d >> 1][(d & 1) * 2 + c] * inv, A.E - 127);
                *reinterpret_cast<uint2*>(a.out + at * D + 32 * b + 4 * g) =
                    make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
              }
              if (a.lse && g == 0) a.lse[at] = l == 0.f ? -INFINITY : (A.m[nt][c] == -INFINITY ? l : (A.m[nt][c] + lg2(l)) * 0.6931471805599453f);
            }
          }
      } else {
        // a run's last piece goes to its drained ring, a first one to the stash
        const bool last = i >= n_units;
        float* dst = last ? reinterpret_cast<float*>(ring) : stash;
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = nt * 8 + 2 * t + c;
#pragma unroll
            for (int b = 0; b < NB; ++b)
              *reinterpret_cast<float4*>(dst + col * (D + 4) + 32 * b + 4 * g) =
                  make_float4(A.o[nt][b][0][c], A.o[nt][b][0][2 + c], A.o[nt][b][1][c], A.o[nt][b][1][2 + c]);
            if (g == 0) {
              dst[COLS * (D + 4) + col] = A.m[nt][c];
              dst[COLS * (D + 4) + COLS + col] = A.l[nt][c];
            }
          }
        if (lane == 0) ph[warp][last ? 1 : 0] = PartHead{item, q.ng, cr, pair, 0, A.E, 0};
      }
    }
    if (!alive) {
      // a copy did not arrive in time: wait (bounded) for those in flight, leave no piece
      for (int k = i; k < min(i + S, n_units); ++k) mbar_wait(&bar[k % S], (k / S) & 1, a.status, kKvWaitNs);
      __syncwarp();
      if (lane == 0) ph[warp][0].units = ph[warp][1].units = 0;
    }
  }
  __syncthreads();

  // ---------------------------------------------------------------- pieces of one CTA
  for (int k = 0; k < 2 * W;) {
    if (ph[k >> 1][k & 1].units == 0) {
      ++k;
      continue;
    }
    const PartHead h = ph[k >> 1][k & 1];
    int e = k + 1;
    while (e < 2 * W && (ph[e >> 1][e & 1].units == 0 || ph[e >> 1][e & 1].item == h.item)) ++e;
    auto piece = [&](int x) {
      return reinterpret_cast<const float*>(x & 1 ? smem + (x >> 1) * C::kRingBytes
                                                  : smem + W * C::kRingBytes + (x >> 1) * C::kStash);
    };
    const bool whole = h.item >= cta_lo && h.item + h.units <= cta_hi;
    int E = 0;
    for (int x = k; x < e; ++x)
      if (ph[x >> 1][x & 1].units) E = max(E, ph[x >> 1][x & 1].E);
    const int slot = h.item <= cta_lo ? 0 : 1;
    float* part = p.parts + (2ll * blockIdx.x + slot) * part_floats(COLS, D);
    const Req q = request<COLS>(p, h.r);
    const int kvh = h.pair / q.rt, rt = h.pair - kvh * q.rt;
    for (int y = tid; y < COLS * (D / 4); y += C::kThreads) {
      const int col = y / (D / 4), d = (y % (D / 4)) * 4;
      float m = -INFINITY, l = 0.f;
      for (int x = k; x < e; ++x)
        if (ph[x >> 1][x & 1].units) m = fmaxf(m, piece(x)[COLS * (D + 4) + col]);
      const float mb = m == -INFINITY ? 0.f : m;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = k; x < e; ++x) {
        const PartHead& hx = ph[x >> 1][x & 1];
        if (!hx.units) continue;
        const float* pc = piece(x);
        const float w = ex2(pc[COLS * (D + 4) + col] - mb);
        l += pc[COLS * (D + 4) + COLS + col] * w;
        const float4 v = *reinterpret_cast<const float4*>(pc + col * (D + 4) + d);
        const int de = hx.E - E;
        o.x += mul_pow2(v.x * w, de);
        o.y += mul_pow2(v.y * w, de);
        o.z += mul_pow2(v.z * w, de);
        o.w += mul_pow2(v.w * w, de);
      }
      if (whole) {
        const int c = rt * COLS + col;
        if (c < q.ql * p.G) {
          const int row = c / p.G, hq = kvh * p.G + c - row * p.G;
          const size_t at = (size_t)(q.qb + row) * a.Hq + hq;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          *reinterpret_cast<uint2*>(a.out + at * D + d) =
              make_uint2(f32x2_to_bf16x2(mul_pow2(o.x * inv, E - 127), mul_pow2(o.y * inv, E - 127)),
                         f32x2_to_bf16x2(mul_pow2(o.z * inv, E - 127), mul_pow2(o.w * inv, E - 127)));
          if (a.lse && d == 0) a.lse[at] = l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + lg2(l)) * 0.6931471805599453f);
        }
      } else {
        *reinterpret_cast<float4*>(part + col * D + d) = o;
        if (d == 0) {
          part[COLS * D + col] = m;
          part[COLS * D + COLS + col] = l;
        }
      }
    }
    if (!whole && tid == 0)
      p.heads[2 * blockIdx.x + slot] =
          PartHead{h.item, h.units, h.r, h.pair, h.item >= cta_lo && h.item + h.units > cta_hi ? 1 : 0, E, 0};
    k = e;
  }
}

// Items cut between CTAs: block (c, col) joins row ``col`` of the item that
// starts in CTA c and ends in a later one, from the parts of every CTA it
// reaches, in order.
template <int D, int NT>
__global__ void __launch_bounds__(128) kv_merge_kernel(const StreamParams p) {
  using C = StreamCfg<D, NT>;
  constexpr int COLS = C::kCols, W = C::kWarps, L = D / 4;  // L lanes of 4 dims
  constexpr int kTeams = 128 / L;
  __shared__ float4 so[kTeams][L];
  __shared__ float sl[kTeams];
  const KvAttnArgs& a = p.a;
  grid_dep_wait();
  const long long U = p.plan[0], A_w = p.plan[1];
  const int c0 = blockIdx.x, col = blockIdx.y;
  PartHead h = p.heads[2 * c0];
  int slot0 = 0;
  if (h.units == 0 || !h.starts) {
    h = p.heads[2 * c0 + 1];
    slot0 = 1;
  }
  if (h.units == 0 || !h.starts) return;
  const Req q = request<COLS>(p, h.r);
  const int kvh = h.pair / q.rt, rt = h.pair - kvh * q.rt;
  const int cc = rt * COLS + col;
  if (cc >= q.ql * p.G) return;
  // last CTA: owner of the item's last unit
  const long long u = h.item + h.units - 1;
  const int c1 = (int)((((u + 1) * A_w - 1) / U) / W);
  auto head_of = [&](int c) { return p.heads[2 * c + (c == c0 ? slot0 : 0)]; };
  auto part_of = [&](int c) { return p.parts + (2ll * c + (c == c0 ? slot0 : 0)) * part_floats(COLS, D); };
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  int E = 0;
  for (int c = c0 + lane; c <= c1; c += 32) {
    m = fmaxf(m, part_of(c)[COLS * D + col]);
    E = max(E, head_of(c).E);
  }
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  E = __reduce_max_sync(0xffffffffu, E);
  const float mb = m == -INFINITY ? 0.f : m;
  const int team = threadIdx.x / L, x = threadIdx.x % L;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0 + team; c <= c1; c += kTeams) {
    const float* pc = part_of(c);
    const float w = ex2(pc[COLS * D + col] - mb);
    l += pc[COLS * D + COLS + col] * w;
    const float4 v = *reinterpret_cast<const float4*>(pc + col * D + 4 * x);
    const int de = head_of(c).E - E;
    o.x += mul_pow2(v.x * w, de);
    o.y += mul_pow2(v.y * w, de);
    o.z += mul_pow2(v.z * w, de);
    o.w += mul_pow2(v.w * w, de);
  }
  so[team][x] = o;
  if (x == 0) sl[team] = l;
  __syncthreads();
  if (team == 0) {
    for (int k = 1; k < kTeams; ++k) {
      const float4 v = so[k][x];
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
      l += sl[k];
    }
    const int row = cc / p.G, hq = kvh * p.G + cc - row * p.G;
    const size_t at = (size_t)(q.qb + row) * a.Hq + hq;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(a.out + at * D + 4 * x) =
        make_uint2(f32x2_to_bf16x2(mul_pow2(o.x * inv, E - 127), mul_pow2(o.y * inv, E - 127)),
                   f32x2_to_bf16x2(mul_pow2(o.z * inv, E - 127), mul_pow2(o.w * inv, E - 127)));
    if (a.lse && x == 0) a.lse[at] = l == 0.f ? -INFINITY : (m == -INFINITY ? l : (m + lg2(l)) * 0.6931471805599453f);
  }
}

template <int D, int NT>
cudaError_t launch_stream(const StreamParams& p, cudaStream_t s) {
  using C = StreamCfg<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv_stream_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = p.max_ctas;
  e = launch_kernel(kv_stream_kernel<D, NT>, dim3(grid), dim3(C::kThreads), C::kSmem, s, false, false, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_merge_kernel<D, NT>, dim3(grid, C::kCols), dim3(128), 0, s, true, false, p);
}

constexpr int kMaxStreamCtas = 256;

}  // namespace

// Workspace of the streaming kernels: plan, part headers, parts (sized for 16 rows).
size_t kv_stream_workspace(int D) {
  return 256 + sizeof(PartHead) * 2 * kMaxStreamCtas + 4 * part_floats(16, D) * 2 * kMaxStreamCtas;
}

cudaError_t launch_kv_stream(const KvAttnArgs& a, int row_limit, int tiles, uint8_t* ws, cudaStream_t s) {
  StreamParams p{};
  p.a = a;
  p.G = a.Hq / a.cache.heads;
  p.row_limit = row_limit;
  p.max_ctas = a.num_sms < kMaxStreamCtas ? a.num_sms : kMaxStreamCtas;
  p.plan = reinterpret_cast<long long*>(ws);
  p.heads = reinterpret_cast<PartHead*>(ws + 256);
  p.parts = reinterpret_cast<float*>(ws + 256 + sizeof(PartHead) * 2 * kMaxStreamCtas);
  if (a.cache.D == 128) return tiles == 1 ? launch_stream<128, 1>(p, s) : launch_stream<128, 2>(p, s);
  return tiles == 1 ? launch_stream<64, 1>(p, s) : launch_stream<64, 2>(p, s);
}

}  // namespace moe

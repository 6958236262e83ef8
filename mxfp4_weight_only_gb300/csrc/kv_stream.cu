// Attention over the 4-bit KV cache, few query rows per request: the cache is
// streamed once (kv_mxfp4_attention, decode and short drafts).
//
// Measured: 256 requests of up to 8192 keys, 28 / 4 heads of 128: 73 us, 3.8 TB/s
// (56 % of the copy rate), bound by the issue of the exact conversions (61 % of
// the slots, 54 % of the ALU pipe); 2 requests of 262,139 keys, 32 / 2 heads: 62 us;
// one of 1,000 keys: 12.3 us, latency.
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
// shuffles).  Queries enter as f16 scaled by a power of two per row (exact down to
// 2^-31 of the row's largest; see kQueryExp), keys as f16 (exact).  Weights enter as the sum of two bf16
// (16 bits, two MMAs: the tensor pipe has room), which keeps a weight of any
// size where the heavier keys' values are zero (one f16 weight, 11 bits, loses
// those below 2^-32; one bf16 weight has 8 bits).  Value scales outside
// 2^-63 .. 2^64 (or NaN bytes) take an exact float32 path (add_group_f32).
//
// Work: a unit is one record of one item (request, kv head, row tile).  All items
// in order, each at the cost of its units and kItemCost more (its queries and
// its result), are cut into equal runs, one per warp of a one-CTA-per-SM grid,
// so ragged batches balance without a host-side plan: every CTA finds its place
// by a prefix sum over the requests.  Each warp streams its
// run through a private ring of bulk copies (one per record) without any
// barrier with other warps.  Items cut between warps are merged in shared
// memory, items cut between CTAs through the workspace by kv_merge_kernel.
#include <type_traits>

#include "common.cuh"
#include "kv_internal.h"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT>
struct StreamCfg {
  static constexpr int NB = D / 32;
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRec = 17 * D;
  static constexpr int kStages = (NT == 1 ? 4 : 8) * (128 / D);  // a power of two, at most 32
  static constexpr int kStep = 2;                                // records per softmax step
  static constexpr int kCols = 8 * NT;
  // a piece in shared memory: O [kCols][D + 4] float, m, l [kCols], reference scale E
  static constexpr int kPieceFloats = kCols * (D + 4) + 2 * kCols + 4;
  static constexpr int kRingBytes = kStages * kRec;
  static constexpr int kStash = kPieceFloats * 4;
  static_assert(kStash <= kRingBytes, "a warp's last piece is stored in its drained ring");
  static constexpr int kSmem = kWarps * (kRingBytes + kStash);
};

// Weights are 2^(S f - m f) with the product S f unrounded and m f rounded, so the
// largest is 2^r with r up to half a unit in the last place of m f: 2^4 at this
// size.  Beyond, both products are rounded (largest weight 1), and taken by a
// quarter: units of log2 would leave float32 before the scores do.
constexpr float kFar = 0x1p28f;
// Plain steps take shifts of the key scales up to this either way: bytes of 64 ..
// 191 stay within 1 .. 254.
constexpr int kPlainShift = 56;

// What an item costs beside its units, in units.  Measured (us at 2 / 4 / 6 / 8 /
// 16): 256 requests, 4 kv heads, up to 8192 keys 77.5 / 75.7 / 74.5 / 75.1 / 78.2;
// 32 of them 23.6 / 22.4 / 22.0 / 21.9 / 23.3; 16 requests x 32 heads of 64, window
// 1024 21.0 / 21.0 / 19.6 / 20.0 / 20.4.
constexpr int kItemCost = 6;
// Least run of a warp, in units: shorter runs only add pieces to merge (1 request
// of 1,000 keys: 12.2 us at 2, 13.6 at 4).
constexpr int kMinRun = 2;

// A piece of an item: one warp's (shared memory) or one CTA's (workspace).
struct PartHead {
  long long item;  // the item's first unit, counted over all items
  int units;       // units of the item; 0: no piece here
  int qb, rows;    // first query row of the request; its rows (query rows x heads)
  int hq0, col0;   // first query head; first row of the row tile
  int starts;      // workspace: 1 = the item starts in this CTA and ends in a later one
  int last_cta;    // the CTA of its last unit
  int E;           // O is in units of 2^(E - 127)
};

__host__ __device__ constexpr size_t part_floats(int cols, int D) { return (size_t)cols * D + 2 * cols; }

struct StreamParams {
  KvAttnArgs a;
  int G;           // query heads per kv head
  int row_limit;   // requests with more rows than this are not this kernel's,
  const int32_t* odd;  // unless marked here ([R], or null: none)
  int max_ctas;
  PartHead* heads;   // [grid][2]
  float* parts;      // [grid][2][part_floats]
};

// What a request asks for: rows, the record range any of its rows can see.
struct Req : KvRequest {
  int glo, ng, rt;
  __device__ __forceinline__ int items(int heads) const { return ng > 0 ? heads * rt : 0; }
};

// a / b, a % b for b >= 1; 32-bit where a allows.
__device__ __forceinline__ long long divmod(long long a, int b, int& rem) {
  if ((a >> 32) == 0) {
    const uint32_t q = (uint32_t)a / (uint32_t)b;
    rem = (int)((uint32_t)a - q * (uint32_t)b);
    return q;
  }
  const long long q = a / b;
  rem = (int)(a - q * b);
  return q;
}

template <int COLS>
__device__ __forceinline__ Req request(const StreamParams& p, int r) {
  const KvAttnArgs& a = p.a;
  Req q;
  static_cast<KvRequest&>(q) = kv_request(a, r);
  const long long rows = (long long)max(q.ql, 0) * p.G;
  const bool mine = rows > 0 && (rows <= p.row_limit || (p.odd && p.odd[r] != 0));
  q.rt = mine ? (int)((rows + COLS - 1) / COLS) : 0;
  q.glo = kv_first_key(q.first, a.window) >> 4;
  const int hi = a.causal ? min(q.n, max(0, q.first + q.ql)) : q.n;  // keys past the last row's are not looked at
  q.ng = mine ? ((hi + 15) >> 4) - q.glo : 0;
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

// A score (or reference) v times its factor f, in units of 4 log2.
__device__ __forceinline__ float quarter(float v, float f) { return __fmul_rn(v, 0.25f * f); }

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

// A token's NB scale bytes in a word (NB = 2: twice).
template <int NB>
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p, int tok) {
  if (NB == 4) return *reinterpret_cast<const uint32_t*>(p + 4 * tok);
  const uint32_t v = *reinterpret_cast<const uint16_t*>(p + 2 * tok);
  return v | (v << 16);
}

// The scale words of tokens tok and tok + 1 (tok even).
template <int NB>
__device__ __forceinline__ void scale_word2(const uint8_t* p, int tok, uint32_t& a, uint32_t& b) {
  if (NB == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + 4 * tok);
    a = u.x;
    b = u.y;
  } else {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p + 2 * tok);
    a = prmt(u, 0u, 0x1010u);
    b = prmt(u, 0u, 0x3232u);
  }
}

// 2^(s-127) of the two bytes of each half of ``w``: bf16 pairs, exact (255: NaN).
__device__ __forceinline__ void e8m0x4_to_bf16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.bf16x2.ue8m0x2 %0, l;\n cvt.rn.bf16x2.ue8m0x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Top bit of a byte set where the byte lies in 64 .. 191 (its two top bits differ).
__device__ __forceinline__ uint32_t usual(uint32_t w) { return w ^ (w << 1); }

// Key scale bytes plus ``shift`` (255 stays), within 0 .. 254: for factors beyond kPlainShift.
__device__ __noinline__ uint32_t shifted_scales(uint32_t w, int shift) {
  uint32_t r = 0;
  for (int b = 0; b < 4; ++b) {
    const int x = (w >> (8 * b)) & 255;
    r |= (uint32_t)(x == 255 ? 255 : min(max(x + shift, 0), 254)) << (8 * b);
  }
  return r;
}

// Any byte of a word outside 64 .. 191 and not 0?
__device__ __forceinline__ bool unusual_scale(uint32_t w) {
  bool r = false;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t x = (w >> (8 * b)) & 255u;
    r |= x != 0u && x - 64u > 127u;
  }
  return r;
}

// Any byte equal to 255?
__device__ __forceinline__ bool has_nan_byte(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u) != 0u;
}

// Largest byte of a word, 255 excluded.
__device__ __forceinline__ int largest_scale(uint32_t w) {
  int m = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int x = (w >> (8 * b)) & 255;
    if (x != 255) m = max(m, x);
  }
  return m;
}

// One item's state in a warp.  Lane (g, t) = (lane / 4, lane % 4) holds, for its
// two rows 2t, 2t+1 of each row tile of 8, dims 4g .. 4g+3 of every block.
template <int D, int NT>
struct Acc {
  static constexpr int NB = D / 32;
  float o[NT][NB][2][4];  // [tile][block][dims 01 / 23][dim a rows 2t, 2t+1; dim b rows 2t, 2t+1]
  float m[NT][2], l[NT][2];  // reference of the scores (before the factor f), sum of weights
  float mf[NT][2];           // m f, 0 while m is -inf
  int E;                     // O is in units of 2^(E - 127)
};

// O += p V in float32 for one record, any value scales (the exceptional case):
// the weights of token k come from the lane that holds them.
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

// The scores of one record in float32 from the queries themselves, in the units of
// the MMAs' (times 2^(shift - e) of each row): for rows whose elements f16 cannot
// hold beside keys large enough to tell.  Lane (g, t): tokens g, g + 8, rows 2t,
// 2t + 1 of each tile.
template <int D, int NT>
__device__ __noinline__ void scores_f32(const KvAttnArgs& a, const uint8_t* rec, int lane, int qb, int rows, int col0, int kvh,
                                        int G, int shift, float (&sc)[NT][4]) {
  constexpr int NB = D / 32;
  const int g = lane >> 2, t = lane & 3;
  for (int i = 0; i < 2 * NT; ++i) {
    const int c = col0 + (i >> 1) * 8 + 2 * t + (i & 1);
    float s[2] = {0.f, 0.f};
    if (c < rows) {
      const int row = c / G;
      const uint16_t* q = a.q + (size_t)(qb + row) * a.q_stride + (size_t)(kvh * G + c - row * G) * D;
      KvQueryRange range;
      for (int k = 0; k < D / 2; ++k) range.add(__ldg(reinterpret_cast<const uint32_t*>(q) + k));
      const int e = kv_query_exp(range.most());
      if (!kv_query_finite(range.most())) s[0] = s[1] = __uint_as_float(0x7FC00000u);
      for (int b = 0; b < NB; ++b) {
        float d[2] = {0.f, 0.f};  // times 2^-8: sums of 32 products stay below 2^128
        for (int k = 0; k < 16; ++k) {  // two elements: row byte 16 b + k
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q) + 16 * b + k);
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4];
            e2m1x8_to_f16x8(rec[(((h * 8 + g) * 4 + (k >> 2)) * NB + b) * 4 + (k & 3)], x[0], x[1], x[2], x[3]);
            d[h] = fmaf(bf16_lo(w) * 0x1p-8f, f16_lo(x[0]), d[h]);
            d[h] = fmaf(bf16_hi(w) * 0x1p-8f, f16_hi(x[0]), d[h]);
          }
        }
        for (int h = 0; h < 2; ++h)
          s[h] += mul_pow2(d[h], (int)rec[16 * D + (8 * h + g) * NB + b] - 127 + shift - e + 8);
      }
    }
    const bool neg = a.scale < 0.f;
    sc[i >> 1][i & 1] = neg ? -s[0] : s[0];
    sc[i >> 1][2 + (i & 1)] = neg ? -s[1] : s[1];
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Dims d .. d + 3 of output row ``row`` (token x query head): O (units of 2^(E - 127)) over the sum of weights.
template <int D>
__device__ __forceinline__ void store4(const KvAttnArgs& a, size_t row, int d, const float4& o, float l, int E) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (E != 127) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mul_pow2(v[k], E - 127);
  }
  *reinterpret_cast<uint2*>(a.out + row * D + d) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
}

// lse from the sum of weights and their reference m (units of 4 log2).
__device__ __forceinline__ void store_lse(const KvAttnArgs& a, size_t row, float l, float m) {
  if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : m == -INFINITY ? l : fmaf(m, 2.772588722239781f, lg2(l) * 0.6931471805599453f);
}

template <int D, int NT>
__global__ void __launch_bounds__(StreamCfg<D, NT>::kThreads, 1) kv_stream_kernel(const StreamParams p) {
  using C = StreamCfg<D, NT>;
  constexpr int NB = C::NB, W = C::kWarps, S = C::kStages, REC = C::kRec, COLS = C::kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W * S];
  __shared__ long long scan_c[W], scan_u[W];
  __shared__ long long before_c[C::kThreads], before_u[C::kThreads];  // cost and units before each request of a chunk
  __shared__ int n_empty, empties[C::kThreads];
  // where each warp's run starts ([W]: where the last one ends): request, item
  // within it, unit within that; units before it; cost before its request
  __shared__ int at_r[W + 1], at_item[W + 1], at_g[W + 1];
  __shared__ long long at_unit[W + 1], at_cost[W + 1];
  __shared__ PartHead ph[2 * W];  // pieces left by each warp: its first, its last
  const KvAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRingBytes;
  float* stash = reinterpret_cast<float*>(smem + W * C::kRingBytes + warp * C::kStash);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&bars[warp * S + s], 1 + a.wait.extra_waiters);
    fence_barrier_init();
    ph[2 * warp].units = ph[2 * warp + 1].units = 0;
  }
  __syncwarp();  // other lanes arrive on the barriers: shuffles and votes order no memory
  if (tid < 2) p.heads[2 * blockIdx.x + tid].units = 0;
  grid_dep_launch_dependents();

  // ---------------------------------------------------------------- cost and units of all requests
  const int H = a.cache.heads;
  // Up to 32 requests every warp finds its own place, one request a lane, and the
  // CTA does not meet before its pieces are merged; beyond, the CTA's threads scan
  // the requests together, a chunk at a time.
  const bool few = a.R <= 32;
  const int chunks = few ? 1 : (a.R + C::kThreads - 1) / C::kThreads;
  long long T = 0, U = 0;          // totals so far
  long long first_c = 0, first_u = 0;  // before this thread's request of the last chunk scanned
  Req mine{};
  auto scan = [&](int ch) {
    const int r = few ? lane : ch * C::kThreads + tid;
    mine = Req{};
    if (r < a.R) mine = request<COLS>(p, r);
    const long long it = mine.items(H), c = it * (mine.ng + kItemCost), u = it * mine.ng;
    long long ic = c, iu = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long xc = __shfl_up_sync(0xffffffffu, ic, o), xu = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) {
        ic += xc;
        iu += xu;
      }
    }
    first_c = T + ic - c;
    first_u = U + iu - u;
    if (few) {
      T = __shfl_sync(0xffffffffu, ic, 31);
      U = __shfl_sync(0xffffffffu, iu, 31);
      return;
    }
    __syncthreads();  // the previous chunk's sums have been read
    if (lane == 31) {
      scan_c[warp] = ic;
      scan_u[warp] = iu;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const long long xc = scan_c[w], xu = scan_u[w];
      if (w < warp) {
        first_c += xc;
        first_u += xu;
      }
      T += xc;
      U += xu;
    }
  };
  // requests without a key: their rows are zeros, written by one CTA each
  auto zero_rows = [&](int r) {
    const Req q = request<COLS>(p, r);
    const long long rows = (long long)q.ql * a.Hq;
    uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)q.qb * a.Hq * D);
    for (long long i = tid; i < rows * (D / 8); i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (long long i = tid; i < rows; i += C::kThreads) a.lse[(size_t)q.qb * a.Hq + i] = -INFINITY;
  };
  for (int ch = 0; ch < chunks; ++ch) {
    if (!few && tid == 0) n_empty = 0;
    scan(ch);
    const bool empty = mine.rt > 0 && mine.ng <= 0;
    if (few) {
      for (uint32_t m = __ballot_sync(0xffffffffu, empty && lane % gridDim.x == blockIdx.x); m; m &= m - 1)
        zero_rows(__ffs(m) - 1);
    } else {
      if (empty && tid % gridDim.x == blockIdx.x) empties[atomicAdd(&n_empty, 1)] = ch * C::kThreads + tid;
      __syncthreads();
      for (int k = 0; k < n_empty; ++k) zero_rows(empties[k]);
      __syncthreads();
    }
  }
  if (U == 0) return;
  // equal runs of cost: the first ``rem`` of A_w warps take one more; few
  // active warps are spread over all CTAs
  const long long cost = T;
  const int A_w = (int)min((long long)gridDim.x * W, (cost + kMinRun - 1) / kMinRun);
  const int wpc = (A_w + gridDim.x - 1) / gridDim.x;  // active warps of a CTA
  int rem;
  const long long per = divmod(cost, A_w, rem);
  auto begin_of = [&](int w) { return w >= A_w ? cost : w * per + min(w, rem); };
  auto cta_of = [&](long long c) {  // the CTA in whose run cost index c lies
    const long long cut = rem * (per + 1);
    int x;
    return (int)(c < cut ? divmod(c, (int)(per + 1), x) : rem + divmod(c - cut, (int)per, x)) / wpc;
  };
  const int gw0 = blockIdx.x * wpc;
  if (gw0 >= A_w) return;
  // where cost index b lies, counted from request r (cost fc and units fu before it);
  // the end of everything counts as after the last unit
  auto place = [&](long long b, int ng, long long fc, long long fu, int& item, int& unit, long long& units) {
    int x;
    item = (int)divmod(min(b, cost - 1) - fc, ng + kItemCost, x);
    unit = max(0, x - kItemCost) + (b == cost ? 1 : 0);
    units = fu + (long long)item * ng + unit;
  };
  int br, citem, cg;  // this warp's run: request, item within it, unit within that
  long long ccost, u_lo, u_hi;  // cost before that request; units before the run and before its end
  if (few) {
    auto find = [&](long long b, int& r, int& item, int& unit, long long& fc, long long& units) {
      // the last request that costs anything and starts at or before b
      r = 31 - __clz(__ballot_sync(0xffffffffu, mine.items(H) > 0 && first_c <= min(b, cost - 1)));
      fc = __shfl_sync(0xffffffffu, first_c, r);
      place(b, __shfl_sync(0xffffffffu, mine.ng, r), fc, __shfl_sync(0xffffffffu, first_u, r), item, unit, units);
    };
    int xr, xi, xg;
    long long xc;
    find(begin_of(gw0 + min(warp, wpc)), br, citem, cg, ccost, u_lo);
    find(begin_of(gw0 + min(warp + 1, wpc)), xr, xi, xg, xc, u_hi);
    if (lane == 0 && warp == 0) at_unit[0] = u_lo;
    if (lane == 0 && warp == wpc - 1) at_unit[wpc] = u_hi;
  } else {
    // thread w finds where warp w's run starts (wpc: where the last one ends)
    for (int ch = 0; ch < chunks; ++ch) {
      if (chunks > 1) {
        if (ch == 0) T = U = 0;
        scan(ch);
      }
      before_c[tid] = first_c;
      before_u[tid] = first_u;
      __syncthreads();
      if (tid <= wpc) {
        const long long b = begin_of(gw0 + tid), in = min(b, cost - 1);
        const int n = min(C::kThreads, a.R - ch * C::kThreads);
        if (in >= before_c[0] && in < T) {  // (T: the cost up to this chunk's end)
          int lo = 0, hi = n;  // before_c[lo] <= in, the last such: requests that cost nothing share a value
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before_c[mid] <= in) lo = mid;
            else hi = mid;
          }
          at_r[tid] = ch * C::kThreads + lo;
          at_cost[tid] = before_c[lo];
          place(b, request<COLS>(p, at_r[tid]).ng, before_c[lo], before_u[lo], at_item[tid], at_g[tid], at_unit[tid]);
        }
      }
      __syncthreads();
    }
    const int w = min(warp, wpc);
    br = at_r[w];
    citem = at_item[w];
    cg = at_g[w];
    ccost = at_cost[w];
    u_lo = at_unit[w];
    u_hi = at_unit[min(warp + 1, wpc)];
  }

  // ---------------------------------------------------------------- this warp's run
  const int n_units = (int)(u_hi - u_lo);
  if (n_units > 0) {
    // record addresses, 32 units at a time, one per lane; null for a page outside the cache
    Req q = request<COLS>(p, br);
    int cr = br;
    long long bo = (long long)citem * q.ng + cg;  // units of request br before the next batch
    auto addresses = [&](int i0) -> const uint8_t* {
      const uint8_t* ptr = nullptr;
      int r = br;
      long long off = bo + lane;
      if (i0 + lane < n_units) {
        Req q = request<COLS>(p, r);
        long long u = (long long)q.items(H) * q.ng;
        while (off >= u) {
          off -= u;
          q = request<COLS>(p, ++r);
          u = (long long)q.items(H) * q.ng;
        }
        int gi;
        const int item = (int)divmod(off, q.ng, gi);
        const int tok = (q.glo + gi) << 4;
        const int pg = a.table[(size_t)r * a.max_blocks + (tok >> a.cache.page_shift)];
        if (pg >= 0 && pg < a.cache.num_pages)
          ptr = a.cache.data + a.cache.record(pg, item / q.rt, (tok & ((1 << a.cache.page_shift) - 1)) >> 4);
      }
      // the next 32 start after lane 31's
      br = __shfl_sync(0xffffffffu, r, 31);
      bo = __shfl_sync(0xffffffffu, off, 31) + 1;
      return ptr;
    };
    const uint64_t policy = l2_policy_evict_first();
    const uint8_t* cur = addresses(0);
    const uint8_t* nxt = nullptr;
    uint32_t here = __ballot_sync(0xffffffffu, cur != nullptr);  // which of the 32 have a record
    uint64_t* bar = bars + warp * S;
    // copies of the units i0 .. i0 + n - 1 (at most 32): each by the lane that holds its address
    auto issue = [&](int i0, int n, int batch) {
      const int d = (lane - i0) & 31, i = i0 + d;
      if (d < n && i < n_units) {
        const uint8_t* src = (i >> 5) == batch ? cur : nxt;
        const uint32_t st = (uint32_t)i % S;
        if (src) {
          mbar_arrive_expect_tx(&bar[st], REC);
          bulk_g2s(ring + st * REC, src, REC, &bar[st], policy);
        } else {
          mbar_arrive(&bar[st]);
        }
      }
    };
    issue(0, S, 0);
    if (n_units > 32) nxt = addresses(32);

    bool alive = true;
    int i = 0;
    while (i < n_units && alive) {
      // ------------------------------------------------------------ next item
      while (citem >= q.items(H)) {
        ccost += (long long)q.items(H) * (q.ng + kItemCost);
        q = request<COLS>(p, ++cr);
        citem = 0;
      }
      const int g0 = cg;
      const int kvh = citem / q.rt, rt = citem - kvh * q.rt;
      const int len = min(q.ng - g0, n_units - i);
      const long long item = u_lo + i - g0;
      // queries: f16 times a power of two per row; f folds scale and log2 e
      uint32_t qf[NT][NB][4];
      float f[NT][2];
      int shift = 0;
      // the largest scale byte of keys that the queries' f16 will do for, and plain steps
      int key_top = 255, plain_top;
      {
        const int rows = q.ql * p.G;
        const float fs = fabsf(a.scale) * kLog2e;
        int e[NT], fe = -1000;
        bool bad[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = rt * COLS + nt * 8 + g;
          KvQueryRange range;
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
            for (int k = 0; k < 4; ++k) range.add(w[k]);
          }
          uint32_t most = range.most();
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          e[nt] = kv_query_exp(most);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t w[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              qf[nt][b][k] = f32x2_to_f16x2(mul_pow2(bf16_lo(w[k]), -e[nt]), mul_pow2(bf16_hi(w[k]), -e[nt]));
          }
          if (__any_sync(0xffffffffu, range.loses(most))) {  // rare
            float rest = range.loses(most) ? kQueryRest : 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint32_t w[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                rest += fabsf(mul_pow2(bf16_lo(w[k]), -e[nt]) - f16_lo(qf[nt][b][k])) +
                        fabsf(mul_pow2(bf16_hi(w[k]), -e[nt]) - f16_hi(qf[nt][b][k]));
            }
            rest += __shfl_xor_sync(0xffffffffu, rest, 1);
            rest += __shfl_xor_sync(0xffffffffu, rest, 2);
            key_top = min(key_top, __reduce_min_sync(0xffffffffu, kv_key_top(rest, fs, e[nt])));
          }
          bad[nt] = !kv_query_finite(most);
          // (a negative scale's sign goes into the queries: factors are positive)
          if (a.scale < 0.f) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int k = 0; k < 4; ++k) qf[nt][b][k] ^= 0x80008000u;
          }
          if (c < rows) fe = max(fe, kv_exponent(fs) + e[nt]);
        }
        // the largest factor's power of two goes into the key scales, so that partial sums
        // stay near the scores' size (a quarter of it, in units of log2)
        fe = __reduce_max_sync(0xffffffffu, fe);
        shift = fs > 0.f ? min(max(fe - 2, -126), 126) : 0;
        // keys up to this byte leave scores (f 2^(kQueryExp + 1) 6 D 2^(s - 127) at most) below kFar
        plain_top = min(key_top, 127 + 28 - (kQueryExp + 1) - 3 - 7 - (fe + 1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float v = mul_pow2(fs, e[nt] - shift);
          if (v == 0.f) {  // scores of 0: by the queries, so that hidden keys stay at -inf
            v = 1.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) qf[nt][b][0] = qf[nt][b][1] = qf[nt][b][2] = qf[nt][b][3] = 0u;
          }
          if (bad[nt]) {
#pragma unroll
            for (int b = 0; b < NB; ++b) qf[nt][b][0] = qf[nt][b][1] = qf[nt][b][2] = qf[nt][b][3] = 0x7FFF7FFFu;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            f[nt][k] = __shfl_sync(0xffffffffu, v, 4 * (2 * t + k));
          }
        }
      }
      // keys [lo, hi) that row c of the request sees (rows past the last: all)
      auto sees = [&](int c, int& lo, int& hi) {
        const int pos = q.first + c / p.G;
        const bool real = c < q.ql * p.G;
        hi = real && a.causal ? min(q.n, pos + 1) : q.n;
        lo = real ? kv_first_key(pos, a.window) : 0;
      };
      int lo_max = 0, hi_min = q.n;  // over the tile's rows: the last sees the latest first key, the first the fewest
      {
        int x;
        sees(min(rt * COLS + COLS, q.ql * p.G) - 1, lo_max, x);
        sees(rt * COLS, x, hi_min);
      }

      // plain steps look for key scale bytes above plain_top too: 191 after this
      const uint32_t key_add = lane < 16 && plain_top < 191 ? (uint32_t)(191 - max(plain_top, 127)) * 0x01010101u : 0u;
      const bool plain = plain_top >= 127 && shift >= -kPlainShift && shift <= kPlainShift;
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
        A.mf[nt][0] = A.mf[nt][1] = 0.f;
      }

      bool far = false;  // a reference beyond kFar
      // a score above its limit moves the reference: 8 above it in units of log2
      float limit[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) limit[nt][0] = limit[nt][1] = -INFINITY;

      // one softmax step.  PLAIN: over the records i .. i + kStep - 1, every row
      // sees every key of them, factors and units are the usual ones; without the
      // branches that look after the rest; returns false, with nothing done, where
      // it meets scales of an unusual size (those that could lead beyond kFar among
      // them).  Else over record i, whatever it holds
      // (``live``: it exists).
      auto step = [&](auto plain_tag, int k, bool live) -> bool {
        constexpr bool PLAIN = decltype(plain_tag)::value;
        constexpr int NG = PLAIN ? C::kStep : 1;
        float sc[NG][NT][4];
        uint32_t vsa[NG][2], vsb[NG][2];  // value scales of tokens 2t, 2t+1 (a, b), plus 8
        const uint8_t* rec[NG];
        const int j0 = (q.glo + g0 + k) << 4;
        uint32_t ok = 0x80808080u;
        const int ct = lane & 15;  // the token whose key (lanes 0-15) or value scales this lane looks at
        const int coff = 16 * D + (lane >> 4) * (D / 2);
#pragma unroll
        for (int r = 0; r < NG; ++r) {
          rec[r] = ring + ((uint32_t)(i + r) % S) * REC;
          const int valid = q.n - (j0 + 16 * r);  // tokens of the record that exist (above 16: all)
          // -------------------------------------------------- scores
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[r][nt][0] = sc[r][nt][1] = sc[r][nt][2] = sc[r][nt][3] = 0.f;
          uint32_t kw[2][NB];
          load_words<NB>(rec[r], lane, kw);
          uint32_t ks0 = scale_word<NB>(rec[r] + 16 * D, g), ks1 = scale_word<NB>(rec[r] + 16 * D, g + 8);
          scale_word2<NB>(rec[r] + 16 * D + D / 2, 2 * t, vsa[r][0], vsb[r][0]);
          scale_word2<NB>(rec[r] + 16 * D + D / 2, 2 * t + 8, vsa[r][1], vsb[r][1]);
          uint32_t look = scale_word<NB>(rec[r] + coff, ct);
          if (!PLAIN && (valid < 16 || !live)) {  // what lies past the end, or outside the cache, is not looked at
            const int v = live ? valid : 0;
            if (g >= v) ks0 = 0x7F7F7F7Fu;
            if (g + 8 >= v) ks1 = 0x7F7F7F7Fu;
            if (2 * t >= v) vsa[r][0] = 0x7F7F7F7Fu;
            if (2 * t + 1 >= v) vsb[r][0] = 0x7F7F7F7Fu;
            if (2 * t + 8 >= v) vsa[r][1] = 0x7F7F7F7Fu;
            if (2 * t + 9 >= v) vsb[r][1] = 0x7F7F7F7Fu;
            if (ct >= v) look = 0x7F7F7F7Fu;
          }
          // (from 127 on, plain_top adds 64 at most: what passes 255 lands below 64)
          ok &= usual(PLAIN ? look + key_add : look);
          float unit = 1.f;  // what the scales as float32 still need
          if (PLAIN) {  // (bytes of 64 .. 191: none carries)
            ks0 += (uint32_t)(shift * 0x01010101);
            ks1 += (uint32_t)(shift * 0x01010101);
          } else if (shift < -kPlainShift || shift > kPlainShift) {
            ks0 = shifted_scales(ks0, shift);
            ks1 = shifted_scales(ks1, shift);
          } else {
            unit = exp2_int(shift);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t x[4], y[4];
            e2m1x8_to_f16x8(kw[0][b], x[0], x[1], x[2], x[3]);
            e2m1x8_to_f16x8(kw[1][b], y[0], y[1], y[2], y[3]);
            // byte -> 2^(s-127): 0 gives 0 (for 2^-127); 255 is seen to below
            float s0 = __uint_as_float((b < 3 ? ks0 << (23 - 8 * b) : ks0 >> 1) & 0x7F800000u);
            float s1 = __uint_as_float((b < 3 ? ks1 << (23 - 8 * b) : ks1 >> 1) & 0x7F800000u);
            if (!PLAIN) {  // (finite, so that products of 0 stay 0)
              s0 = fminf(s0 * unit, 3.402823466e38f);
              s1 = fminf(s1 * unit, 3.402823466e38f);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4];
              const float z[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16_16816(d, x[0], y[0], x[1], y[1], qf[nt][b][0], qf[nt][b][1], z);
              mma_f16_16816(d, x[2], y[2], x[3], y[3], qf[nt][b][2], qf[nt][b][3], d);
              sc[r][nt][0] = fmaf(d[0], s0, sc[r][nt][0]);
              sc[r][nt][1] = fmaf(d[1], s0, sc[r][nt][1]);
              sc[r][nt][2] = fmaf(d[2], s1, sc[r][nt][2]);
              sc[r][nt][3] = fmaf(d[3], s1, sc[r][nt][3]);
            }
          }
        }
        if (!PLAIN && key_top < 255) {
          const int v = live ? q.n - j0 : 0;
          const int top = max(g < v ? largest_scale(scale_word<NB>(rec[0] + 16 * D, g)) : 0,
                              g + 8 < v ? largest_scale(scale_word<NB>(rec[0] + 16 * D, g + 8)) : 0);
          if (__reduce_max_sync(0xffffffffu, top) > key_top) {
            float s[NT][4];
            scores_f32<D, NT>(a, rec[0], lane, q.qb, q.ql * p.G, rt * COLS, kvh, p.G, shift, s);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) sc[0][nt][c] = s[nt][c];
          }
        }
        // ---------------------------------------------------- scales of an unusual size
        bool wide = !PLAIN && A.E != 127;
        const bool unusual = __any_sync(0xffffffffu, ok != 0x80808080u);
        if (PLAIN && unusual) return false;
        if (!PLAIN && (unusual || wide)) {
#pragma unroll
          for (int r = 0; r < NG; ++r) {
            const int v = live ? q.n - (j0 + 16 * r) : 0;
            // NaN blocks of keys or values make their token NaN
            const uint8_t* ks = rec[r] + 16 * D;
            const float nan = __uint_as_float(0x7FC00000u);
            const bool n0 = g < v && (has_nan_byte(scale_word<NB>(ks, g)) || has_nan_byte(scale_word<NB>(ks + D / 2, g)));
            const bool n1 = g + 8 < v &&
                            (has_nan_byte(scale_word<NB>(ks, g + 8)) || has_nan_byte(scale_word<NB>(ks + D / 2, g + 8)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (n0) sc[r][nt][0] = sc[r][nt][1] = nan;
              if (n1) sc[r][nt][2] = sc[r][nt][3] = nan;
            }
            // zero value scales are as good as usual ones: blocks below 2^-124, next to nothing
            const bool odd = unusual_scale(vsa[r][0]) || unusual_scale(vsb[r][0]) || unusual_scale(vsa[r][1]) ||
                             unusual_scale(vsb[r][1]);
            wide |= (bool)__any_sync(0xffffffffu, odd);
            int mx = max(max(largest_scale(vsa[r][0]), largest_scale(vsb[r][0])),
                         max(largest_scale(vsa[r][1]), largest_scale(vsb[r][1])));
            mx = __reduce_max_sync(0xffffffffu, mx);
            // sums (weights up to 2^8, values below 8 2^(mx - 127), q.n keys) have to
            // stay below 2^128 in units of 2^(E - 127); no larger a unit than that, as
            // other blocks and keys may be small
            mx += 11 + 32 - __clz(q.n) - 128;
            if (wide && mx > A.E) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                  for (int c = 0; c < 8; ++c) A.o[nt][b][c >> 2][c & 3] = mul_pow2(A.o[nt][b][c >> 2][c & 3], A.E - mx);
              A.E = mx;
            }
          }
        }
        // ---------------------------------------------------- masks
        if (!PLAIN) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              int lo, hi;
              sees(rt * COLS + nt * 8 + 2 * t + c, lo, hi);
#pragma unroll
              for (int r = 0; r < NG; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int j = j0 + 16 * r + g + 8 * h;
                  if (j >= hi || j < lo || !live) sc[r][nt][2 * h + c] = -INFINITY;
                }
            }
        }
        // ---------------------------------------------------- running maximum and sum
        float mn[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = fmaxf(sc[0][nt][c], sc[0][nt][c + 2]);
#pragma unroll
            for (int r = 1; r < NG; ++r) v = fmaxf(v, fmaxf(sc[r][nt][c], sc[r][nt][c + 2]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            mn[nt][c] = v;
            // the reference follows the maximum only where a weight would pass 2^8
            grow |= v > limit[nt][c];
          }
        if (__any_sync(0xffffffffu, grow)) {
          if (!PLAIN) {
            bool beyond = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float m1 = fmaxf(A.m[nt][c], mn[nt][c]);
                beyond |= m1 != -INFINITY && fabsf(m1 * f[nt][c]) > kFar;
              }
            far |= (bool)__any_sync(0xffffffffu, beyond);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float m1 = fmaxf(A.m[nt][c], mn[nt][c]), mf1 = m1 == -INFINITY ? 0.f : m1 * f[nt][c];
              al[c] = A.m[nt][c] == -INFINITY ? 0.f : ex2(A.mf[nt][c] - mf1);
              if (!PLAIN && far && al[c] != 0.f) al[c] = ex2(4.f * __fsub_rn(quarter(A.m[nt][c], f[nt][c]), quarter(m1, f[nt][c])));
              A.l[nt][c] *= al[c];
              A.m[nt][c] = m1;
              A.mf[nt][c] = mf1;
              limit[nt][c] = m1 == -INFINITY ? m1 : m1 + __fdividef(8.f, f[nt][c]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int c = 0; c < 8; ++c) A.o[nt][b][c >> 2][c & 3] *= al[c & 1];
          }
        }
        uint32_t pt[NG][NT][2][2];  // transposed: [tokens 2t, 2t+1 / plus 8][upper 8 bits / the rest], row g
#pragma unroll
        for (int r = 0; r < NG; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float s = sc[r][nt][c], ff = f[nt][c & 1], m = A.m[nt][c & 1];
              sc[r][nt][c] = ex2(!PLAIN && far ? 4.f * __fsub_rn(quarter(s, ff), m == -INFINITY ? 0.f : quarter(m, ff))
                                               : fmaf(s, ff, -A.mf[nt][c & 1]));
              A.l[nt][c & 1] += sc[r][nt][c];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p0 = sc[r][nt][2 * h], p1 = sc[r][nt][2 * h + 1];
              const uint32_t u = __float_as_uint(p0), v = __float_as_uint(p1);
              pt[r][nt][h][0] = movm(prmt(u, v, 0x7632u));
              pt[r][nt][h][1] =
                  movm(f32x2_to_bf16x2(p0 - __uint_as_float(u & 0xFFFF0000u), p1 - __uint_as_float(v & 0xFFFF0000u)));
            }
          }
        // ---------------------------------------------------- weighted sum
        if (PLAIN || !wide) {
#pragma unroll
          for (int r = 0; r < NG; ++r) {
            uint32_t vw[2][NB], vs[2][NB];  // vs: scales of tokens (2t, 2t+1) as bf16 pairs, per block
            load_words<NB>(rec[r] + 8 * D, lane, vw);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              e8m0x4_to_bf16x4(prmt(vsa[r][h], vsb[r][h], 0x5140u), vs[h][0], vs[h][1]);
              if (NB == 4) e8m0x4_to_bf16x4(prmt(vsa[r][h], vsb[r][h], 0x7362u), vs[h][NB - 2], vs[h][NB - 1]);
            }
#pragma unroll
            for (int bp = 0; bp < NB / 2; ++bp) {
              // [half][block of the pair][dim]: two tokens, one dimension
              uint32_t xv[2][2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) token_pairs(vw[h][bp], vw[h][NB / 2 + bp], xv[h][0], xv[h][1]);
#pragma unroll
              for (int bb = 0; bb < 2; ++bb) {
                const int b = 2 * bp + bb;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int w = 0; w < 2; ++w) {
                    const uint32_t p0 = bf16mul2(pt[r][nt][0][w], vs[0][b]), p1 = bf16mul2(pt[r][nt][1][w], vs[1][b]);
                    mma_bf16_16816(A.o[nt][b][0], xv[0][bb][0], xv[0][bb][1], xv[1][bb][0], xv[1][bb][1], p0, p1);
                    mma_bf16_16816(A.o[nt][b][1], xv[0][bb][2], xv[0][bb][3], xv[1][bb][2], xv[1][bb][3], p0, p1);
                  }
              }
            }
          }
        } else {
          // (copies, so that the common path keeps both in registers)
          Acc<D, NT> B = A;
#pragma unroll
          for (int r = 0; r < NG; ++r) {
            float w[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) w[nt][c] = sc[r][nt][c];
            add_group_f32<D, NT>(B, rec[r], lane, w, live ? q.n - (j0 + 16 * r) : 0);
          }
          A = B;
        }
        return true;
      };

      // waits for the records i .. i + n - 1 (1 or 2)
      auto wait = [&](int n) -> bool {
        const uint32_t s0 = (uint32_t)i % S, p0 = ((uint32_t)i / S) & 1u;
        const uint32_t s1 = (uint32_t)(i + n - 1) % S, p1 = ((uint32_t)(i + n - 1) / S) & 1u;
        return __all_sync(0xffffffffu, mbar_try_wait2(&bar[s0], p0, &bar[s1], p1)) ||
               (mbar_wait_warp(&bar[s0], p0, a.status, a.wait.limit_ns) &&
                mbar_wait_warp(&bar[s1], p1, a.status, a.wait.limit_ns));
      };
      for (int k = 0; k < len && alive;) {
        // plain steps ahead, within this batch of 32 addresses
        int np = 0;
        const int j0 = (q.glo + g0 + k) << 4, in = i & 31;
        if (plain && A.E == 127 && !far && j0 >= lo_max) {
          np = min(min(len - k, 32 - in), (hi_min - j0) >> 4) / C::kStep;
          const uint32_t need = (uint32_t)((1ull << (C::kStep * max(np, 0))) - 1ull) << in;
          if ((here & need) != need) np = 0;
        }
        bool usual_scales = np > 0;
        for (; np > 0; --np) {
          alive = wait(C::kStep);
          if (!alive) break;
          usual_scales = step(std::true_type{}, k, true);
          if (!usual_scales) break;
          // the stages are free: the records S units on
          __syncwarp();
          issue(i + S, C::kStep, i >> 5);
          i += C::kStep;
          k += C::kStep;
        }
        if (!alive) break;
        if (!usual_scales) {
          alive = wait(1);
          if (!alive) break;
          step(std::false_type{}, k, (here >> (i & 31)) & 1u);
          __syncwarp();
          issue(i + S, 1, i >> 5);
          ++i;
          ++k;
        }
        if ((i & 31) == 0) {
          cur = nxt;
          here = __ballot_sync(0xffffffffu, cur != nullptr);
          nxt = i + 32 < n_units ? addresses(i + 32) : nullptr;
        }
      }
      cg = 0;  // the run goes on with the next item
      ++citem;
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
      // from here on m is in units of 4 log2
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (A.m[nt][c] != -INFINITY) A.m[nt][c] = quarter(A.m[nt][c], f[nt][c]);
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
#pragma unroll
              for (int b = 0; b < NB; ++b)
                store4<D>(a, at, 32 * b + 4 * g,
                          make_float4(A.o[nt][b][0][c], A.o[nt][b][0][2 + c], A.o[nt][b][1][c], A.o[nt][b][1][2 + c]),
                          A.l[nt][c], A.E);
              if (g == 0) store_lse(a, at, A.l[nt][c], A.m[nt][c]);
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
        if (lane == 0)
          ph[2 * warp + (last ? 1 : 0)] =
              PartHead{item, q.ng, q.qb, q.ql * p.G, kvh * p.G, rt * COLS, 0,
                       cta_of(ccost + (long long)(citem - 1) * (q.ng + kItemCost) + kItemCost + q.ng - 1), A.E};
      }
    }
    if (!alive) {
      // a copy did not arrive in time: wait (bounded) for those in flight, leave no piece
      for (int k = i; k < min(i + S, n_units); ++k) mbar_wait_warp(&bar[k % S], (k / S) & 1, a.status, a.wait.limit_ns);
      __syncwarp();
      if (lane == 0) ph[2 * warp].units = ph[2 * warp + 1].units = 0;
    }
  }
  __syncthreads();

  const long long cta_lo = at_unit[0], cta_hi = at_unit[wpc];

  // ---------------------------------------------------------------- pieces of one CTA
  // Lane x of every warp looks at piece x (in order of the units): consecutive
  // pieces of one item form a run; a warp takes four rows of one run at a time,
  // eight lanes a row.
  static_assert(2 * W <= 32, "one piece per lane");
  const bool has = lane < 2 * W && ph[min(lane, 2 * W - 1)].units > 0;
  const long long id = has ? ph[lane].item : -1;
  const uint32_t pieces = __ballot_sync(0xffffffffu, has);
  const uint32_t below = pieces & ((1u << lane) - 1u);
  const long long prev = __shfl_sync(0xffffffffu, id, below ? 31 - __clz(below) : lane);
  const uint32_t heads = __ballot_sync(0xffffffffu, has && (!below || prev != id));  // first piece of each run
  auto floats = [&](int x) {
    return reinterpret_cast<const float*>(x & 1 ? smem + (x >> 1) * C::kRingBytes
                                                : smem + W * C::kRingBytes + (x >> 1) * C::kStash);
  };
  constexpr int N = D / 32;  // 16-byte words of a row per lane: word x + 8 d
  const int n_tasks = __popc(heads) * (COLS / 4);
  for (int task = warp; task < n_tasks; task += W) {
    const int col = task % (COLS / 4) * 4 + (lane >> 3), x8 = lane & 7;
    uint32_t at = heads;  // the run's first piece: bit number task / (COLS / 4)
    for (int x = task / (COLS / 4); x; --x) at &= at - 1;
    const int k = __ffs(at) - 1;
    const uint32_t above = heads & ~((2u << k) - 1u);
    const uint32_t run = pieces & (above ? ((1u << (__ffs(above) - 1)) - 1u) : 0xFFFFFFFFu) & ~((1u << k) - 1u);
    const PartHead h = ph[k];
    float m = -INFINITY;
    int E = 0;
    for (uint32_t x = run; x; x &= x - 1) {
      const int y = __ffs(x) - 1;
      m = fmaxf(m, floats(y)[COLS * (D + 4) + col]);
      E = max(E, ph[y].E);
    }
    const float mb = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o[N];
#pragma unroll
    for (int d = 0; d < N; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t x = run; x; x &= x - 1) {
      const int y = __ffs(x) - 1;
      const float* pc = floats(y);
      const float w = ex2(4.f * (pc[COLS * (D + 4) + col] - mb));
      l = fmaf(pc[COLS * (D + 4) + COLS + col], w, l);
      const int de = ph[y].E - E;
#pragma unroll
      for (int d = 0; d < N; ++d) {
        float4 v = *reinterpret_cast<const float4*>(pc + col * (D + 4) + 4 * x8 + 32 * d);
        if (de != 0) v = make_float4(mul_pow2(v.x, de), mul_pow2(v.y, de), mul_pow2(v.z, de), mul_pow2(v.w, de));
        o[d].x = fmaf(v.x, w, o[d].x);
        o[d].y = fmaf(v.y, w, o[d].y);
        o[d].z = fmaf(v.z, w, o[d].z);
        o[d].w = fmaf(v.w, w, o[d].w);
      }
    }
    if (h.item >= cta_lo && h.item + h.units <= cta_hi) {  // whole in this CTA
      const int c = h.col0 + col;
      if (c < h.rows) {
        const int row = c / p.G;
        const size_t dst = (size_t)(h.qb + row) * a.Hq + h.hq0 + c - row * p.G;
#pragma unroll
        for (int d = 0; d < N; ++d) store4<D>(a, dst, 4 * x8 + 32 * d, o[d], l, E);
        if (x8 == 0) store_lse(a, dst, l, m);
      }
    } else {
      const int slot = h.item <= cta_lo ? 0 : 1;
      float* part = p.parts + (2ll * blockIdx.x + slot) * part_floats(COLS, D);
#pragma unroll
      for (int d = 0; d < N; ++d) *reinterpret_cast<float4*>(part + col * D + 4 * x8 + 32 * d) = o[d];
      if (x8 == 0) {
        part[COLS * D + col] = m;
        part[COLS * D + COLS + col] = l;
        if (col == 0) {
          PartHead hh = h;
          hh.starts = h.item >= cta_lo && h.item + h.units > cta_hi ? 1 : 0;
          hh.E = E;
          p.heads[2 * blockIdx.x + slot] = hh;
        }
      }
    }
  }
}

// Items cut between CTAs: block (c, col) joins row ``col`` of the item that
// starts in CTA c and ends in a later one, from the parts of every CTA it
// reaches, in order.
template <int D, int NT>
__global__ void __launch_bounds__(128) kv_merge_kernel(const StreamParams p) {
  using C = StreamCfg<D, NT>;
  constexpr int COLS = C::kCols;
  grid_dep_wait();
  const int c0 = blockIdx.x, col = blockIdx.y;
  PartHead h = p.heads[2 * c0];
  const PartHead h1 = p.heads[2 * c0 + 1];
  int slot0 = 0;
  if (h.units == 0 || !h.starts) {
    h = h1;
    slot0 = 1;
  }
  if (h.units == 0 || !h.starts) return;
  const int cc = h.col0 + col;
  if (cc >= h.rows) return;
  const int c1 = h.last_cta;
  auto slot_of = [&](int c) { return 2ll * c + (c == c0 ? slot0 : 0); };
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  int E = 0;
  for (int c = c0 + lane; c <= c1; c += 32) {
    m = fmaxf(m, p.parts[slot_of(c) * part_floats(COLS, D) + COLS * D + col]);
    E = max(E, p.heads[slot_of(c)].E);
  }
  m = warp_max(m);
  E = __reduce_max_sync(0xffffffffu, E);
  const float mb = m == -INFINITY ? 0.f : m;
  constexpr int L = D / 4, kTeams = 128 / L;  // L lanes of 4 dims take every kTeams-th part
  const int team = threadIdx.x / L, x = threadIdx.x % L;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0 + team; c <= c1; c += kTeams) {
    const float* pc = p.parts + slot_of(c) * part_floats(COLS, D);
    const float w = ex2(4.f * (pc[COLS * D + col] - mb));
    l = fmaf(pc[COLS * D + COLS + col], w, l);
    const float4 v = *reinterpret_cast<const float4*>(pc + col * D + 4 * x);
    const int de = p.heads[slot_of(c)].E - E;
    o.x += mul_pow2(v.x * w, de);
    o.y += mul_pow2(v.y * w, de);
    o.z += mul_pow2(v.z * w, de);
    o.w += mul_pow2(v.w * w, de);
  }
  __shared__ float4 so[kTeams][L];
  __shared__ float sl[kTeams];
  so[team][x] = o;
  if (x == 0) sl[team] = l;
  __syncthreads();
  if (team == 0) {
#pragma unroll
    for (int k = 1; k < kTeams; ++k) {
      const float4 v = so[k][x];
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
      l += sl[k];
    }
    const int row = cc / p.G;
    const size_t dst = (size_t)(h.qb + row) * p.a.Hq + h.hq0 + cc - row * p.G;
    store4<D>(p.a, dst, 4 * x, o, l, E);
    if (x == 0) store_lse(p.a, dst, l, m);
  }
}

template <int D, int NT>
cudaError_t launch_stream(const StreamParams& p, cudaStream_t s) {
  using C = StreamCfg<D, NT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_shared(kv_stream_kernel<D, NT>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const int grid = p.max_ctas;
  e = launch_kernel(kv_stream_kernel<D, NT>, dim3(grid), dim3(C::kThreads), C::kSmem, s, false, false, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv_merge_kernel<D, NT>, dim3(grid, C::kCols), dim3(128), 0, s, true, false, p);
}

constexpr int kMaxStreamCtas = 256;

}  // namespace

// Workspace of the streaming kernels: part headers, parts (sized for 16 rows).
size_t kv_stream_workspace(int D) {
  return sizeof(PartHead) * 2 * kMaxStreamCtas + 4 * part_floats(16, D) * 2 * kMaxStreamCtas;
}

cudaError_t launch_kv_stream(const KvAttnArgs& a, int row_limit, const int32_t* odd, int tiles, uint8_t* ws, cudaStream_t s) {
  StreamParams p{};
  p.a = a;
  p.G = a.Hq / a.cache.heads;
  p.row_limit = row_limit;
  p.odd = odd;
  p.max_ctas = a.num_sms < kMaxStreamCtas ? a.num_sms : kMaxStreamCtas;
  p.heads = reinterpret_cast<PartHead*>(ws);
  p.parts = reinterpret_cast<float*>(ws + sizeof(PartHead) * 2 * kMaxStreamCtas);
  if (a.cache.D == 128) return tiles == 1 ? launch_stream<128, 1>(p, s) : launch_stream<128, 2>(p, s);
  return tiles == 1 ? launch_stream<64, 1>(p, s) : launch_stream<64, 2>(p, s);
}

}  // namespace moe

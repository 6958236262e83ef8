// Attention over the 4-bit KV cache, many query rows per request (prompts):
// tcgen05 MMAs (kv_mxfp4_attention).
//
// Measured: a prompt of 8192 tokens, 28 / 4 heads of 128: 459 us, 1048 TFLOP/s (54 %
// of the library's bf16 matrix product): a tile's chain scores - softmax - product
// is longer than the MMAs of the other tile beside it.
//
// One CTA takes up to 256 rows (query tokens x heads of one kv head, in two
// tiles of 128) of one request and walks over the keys they can see, 128 at a
// time:
//   S = Q K^T          tcgen05 f16, accumulator 128 columns of tensor memory
//   p = 2^(S f - m)    f: scale, log2 e and the row's power of two; m follows the
//                      row's maximum only where p would pass 2^6, so the sum
//                      below is rarely rescaled
//   O += P V           tcgen05 f16, P from tensor memory (over S's columns)
// Eight converter warps expand each 128-key tile of the cache once for both
// query tiles: E2M1 codes to f16 (one conversion per two values) times the
// block's 2^(s-127), exact for scale bytes 104 .. 140 (and 0, blocks below
// 2^-124, as zeros); K rows and V rows go to shared memory as they are, K as the
// K-major and V as the MN-major operand, both with the 128-byte swizzle.  A
// request with any other scale byte (NaN among them), or with scores from kFarScore
// on, is marked and done again by the streaming kernel, which runs next.  Queries
// enter as f16 times a power of two per row (exact down to 2^-31 of the row's
// largest; a row with smaller ones that could tell marks its request: see
// kQueryExp), weights as f16 of p 2^9 (11 bits down to p = 2^-23 of the reference,
// multiples of 2^-33 below), in items with few keys and in those of a shared prefix with
// decoding rows as two bf16 (kFewKeys).
// While one tile's softmax runs, the tensor core works on the other tile.  Each
// query tile has an issuing thread of its own: a thread that issues MMAs keeps
// only a short queue, so its barrier probes and commits (about 100 cycles each)
// leave the tensor core idle unless another thread's MMAs fill in.  The two take
// turns, which keeps one tile's softmax beside the other's MMAs (without turns
// both softmaxes fell into step, and then both products).
#include "common.cuh"
#include "kv_internal.h"

namespace moe {

namespace {

constexpr int kSoftWarps = 8, kConvWarp = 8, kConvWarps = 8, kMmaWarp = 16;
constexpr int kPromptThreads = 32 * (kMmaWarp + 4);  // the last two warps only fill a warpgroup
// Registers a thread of each warpgroup (launched with 96, 61,440 in all): 2
// softmax groups x 128 x 160 + 2 converter groups x 128 x 56 + 128 x 40 = 60,416.
constexpr int kLaunchRegs = 96, kSoftRegs = 160, kConvRegs = 56, kMmaRegs = 40;
static_assert(128 * (2 * kSoftRegs + 2 * kConvRegs + kMmaRegs) <= kPromptThreads * kLaunchRegs, "register split");
constexpr int kKeys = kKvTile;     // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
// Weights are held in f16 times 2^kWeightExp; one may reach 2^kSlack before its
// row's reference moves (at most 2^15 in f16), which rescales O.
constexpr float kSlack = 6.f, kWeightExp = 9.f;
// Where a row sees few keys, all with a value may weigh next to nothing beside
// one without: in items with a row that sees at most this many (its first row
// sees the fewest: short requests and windows, the start of a prompt), weights
// enter as the sum of two bf16 (16 bits at any size, as in the streaming kernel) and V as bf16,
// in two products.  (64 query and 8 kv heads, 256 keys: 32 requests of 64 tokens 70
// us, with one f16 weight 64, in the streaming kernel 225; 16 of 256 tokens 115,
// 105 and 524.)
// So do row tiles of a shared prefix's slices, whatever their keys, with a row of a request that is streamed without a
// prefix, where its weights have 16 bits.  (28 / 4 heads of 128: 64 requests behind 32,768 tokens 87 us, with one
// f16 weight 82; 256 behind 8192 93 and 88.)
constexpr int kFewKeys = 256;
// A weight is off by up to a unit in the last place of its row's reference
// (products S f unrounded, the reference and its sum with kWeightExp rounded): from
// here on by more than f16 has room for above 2^(kSlack + kWeightExp).
constexpr float kFarScore = 0x1p22f;
constexpr int kTopScale = 140;  // the largest scale byte that f16 operands hold

template <int D>
struct PromptCfg {
  static constexpr int kQBytes = 128 * D * 2;            // one query tile
  static constexpr int kTile = kKeys * D * 2;            // one K or V tile
  static constexpr int kStages = 2;
  static constexpr int kKOff = 2 * kQBytes, kVOff = kKOff + kStages * kTile;
  static constexpr int kBarOff = kVOff + kStages * kTile;
  static constexpr int kSmem = 1024 + kBarOff + 256;  // (PromptShared: 160 bytes)
  // tensor memory: S (and P) of both tiles, O of both tiles
  static constexpr uint32_t kSCol = 0, kOCol = 256, kCols = 512;
};

struct PromptParams {
  KvAttnArgs a;
  int G, row_limit;
  int slice_tiles;  // shared prefix: row tiles of a slice at most, 0: its slices are streamed
  bool few_rows;    // shared prefix: no request has more than row_limit rows
  int32_t* odd;  // [R] set for requests with scales outside the exact range
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_alloc(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Matrix descriptor, 128-byte swizzle.  K-major (rows of 64 values of K): groups
// of 8 rows 1024 bytes apart.  MN-major (rows of 64 values of MN, one per K):
// groups of 8 K 1024 bytes apart (stride), next 64 of MN ``lead`` bytes on.
__device__ __forceinline__ uint64_t sw128(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, f16 or bf16 operands, f32 accumulator, M x N; B MN-major with ``tb``.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool tb, bool bf16 = false) {
  return (1u << 4) | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (tb ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The issuing thread must not fall behind the tensor core (an MMA takes 64
// cycles).  Its operands live in uniform registers: the whole warp runs the
// issuing loop on warp-uniform values and one elected lane issues (computed in a
// branch of one lane, every operand is moved there for every MMA: about 120
// cycles an MMA).  Descriptors differ in their low word only, accumulation is a
// constant wherever it can be.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t hi, uint32_t bytes) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
  return d;
}
__device__ __forceinline__ void mma_ss_first(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, 0, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.eq.u32 p, 0, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma_ts_acc(uint32_t d, uint32_t a, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bd, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.eq.u32 p, 0, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bd), "r"(id)
      : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for the loads before it; the registers pass through, so that no use moves above.
__device__ __forceinline__ void tc_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) : : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// a * b + c and a + b on two floats at once.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float mul_pow2(float v, int e) {
  const int c = min(max(e, -252), 252), h = c >> 1;
  return v * exp2_int(h) * exp2_int(c - h);
}

// The f16 factors 2^(s-127), twice each, of a word's first NB scale bytes, for s
// in 104 .. 140 (below 113 subnormal, still exact) and 0 (blocks below 2^-124:
// zeros); any other sets ``odd``.
template <int NB>
__device__ __forceinline__ void scale_pairs(uint32_t w, uint32_t (&f)[4], bool& odd) {
  if (NB == 2) w |= 0x7F7F0000u;
  const uint32_t d = w - 0x70707070u;  // exponent fields s - 112, 1 .. 28 for s in 113 .. 140, if no byte borrows
  const uint32_t e = d << 2;           // upper bytes of the factors
#pragma unroll
  for (int b = 0; b < NB; ++b) f[b] = prmt(e, 0u, 0x0404u | ((uint32_t)b << 4) | ((uint32_t)b << 12));
  if (((d | (d - 0x01010101u) | (d + 0x03030303u)) & 0xE0E0E0E0u) != 0u) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t s = (w >> (8 * b)) & 255u;
      const int x = (int)s - 112;
      const uint32_t v = s == 0u ? 0u : x > 0 ? (uint32_t)min(x, 30) << 10 : 1u << max(x + 9, 0);
      odd |= s != 0u && s - 104u > 36u;
      f[b] = v | (v << 16);
    }
  }
}

// Barriers and flags of a CTA, after its tiles in shared memory.
template <int S>
struct PromptShared {
  uint64_t k_full[S], k_empty[S];  // a K tile is in shared memory; its MMAs are done
  uint64_t v_full[S], v_empty[S];
  uint64_t q_full;     // the query tiles are in shared memory
  uint64_t s_full[2];  // scores of a tile are in tensor memory
  uint64_t p_full[2];  // weights are, and O is in their unit
  uint64_t o_done[2];  // the product with V is done
  uint64_t turn[2];    // the other query tile's MMAs have been issued
  uint64_t drain[2];
  uint32_t tmem_slot;
  volatile int abort_flag;
};

// One item: the rows of request r from row0 on, of kv head kvh.  FEW: see kFewKeys.
// SHARED: the call's requests share a prefix (KvShared); results are sums.
template <int D, bool FEW, bool SHARED = false>
__device__ __forceinline__ void prompt_item(const PromptParams& p, uint8_t* smem, uint32_t tmem, int r, int kvh, int row0,
                                            const KvRequest* known = nullptr) {
  using C = PromptCfg<D>;
  constexpr int NB = D / 32, S = C::kStages;
  PromptShared<S>& sh = *reinterpret_cast<PromptShared<S>*>(smem + C::kBarOff);
  uint64_t *k_full = sh.k_full, *k_empty = sh.k_empty, *v_full = sh.v_full, *v_empty = sh.v_empty, *q_full = &sh.q_full;
  uint64_t *s_full = sh.s_full, *p_full = sh.p_full, *o_done = sh.o_done, *turn = sh.turn, *drain = sh.drain;
  volatile int* abort_flag = &sh.abort_flag;
  const KvAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const KvRequest rq = SHARED ? *known : kv_request<SHARED>(a, r);
  const int qb = rq.qb, ql = rq.ql, n = rq.n;
  const int rows = min(ql * p.G - row0, 256);  // rows of this CTA
  const int first_pos = rq.first + row0 / p.G, last_pos = rq.first + (row0 + rows - 1) / p.G;
  const int key_hi = rq.causal ? min(n, last_pos + 1) : n;
  const int key_lo = kv_first_key(first_pos, a.window);
  const int t0 = key_lo / kKeys, nt = kv_tiles(key_lo, key_hi);
  const int nq = rows > 128 ? 2 : 1;
  const int32_t* table = SHARED && r >= a.R ? a.sh.table : a.table + (size_t)r * a.max_blocks;

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------- softmax: thread = row
    const int x = warp >> 2, quad = warp & 3;
    const int trow = 32 * quad + lane;           // row of the tile
    const int row = row0 + 128 * x + trow;       // row of the request
    const bool real = 128 * x + trow < rows;
    const int i = row / p.G, hq = kvh * p.G + row - i * p.G;
    float f = 1.f;
    {
      // the row's query, f16 times a power of two
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)(qb + i) * a.q_stride + (size_t)hq * D);
      uint4 u[D / 8];
      KvQueryRange range;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) u[c] = real ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) range.add(w[k]);
      }
      const int e = kv_query_exp(range.most());
      const float fs = fabsf(a.scale) * kLog2e;
      f = mul_pow2(fs, e);
      bool held = f < 0x1p100f && kv_query_finite(range.most());  // (f itself may have overflowed)
      // 2^-e in two factors (either alone may leave the range); none where the scores are all 0
      float e0 = exp2_int((-e) >> 1), e1 = exp2_int(-e - ((-e) >> 1));
      if (f == 0.f) {
        f = 1.f;
        e0 = 0.f;
      }
      if (range.loses(range.most())) {  // rare
        float rest = kQueryRest;
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
          const float v = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src) + c) << 16) * e0 * e1;
          rest += fabsf(v - f16_lo(f32x2_to_f16x2(v, 0.f)));
        }
        held = held && kv_key_top(rest, fs, e) >= kTopScale;
      }
      // a row that f16 does not hold is NaN, which marks the request at the end
      if (!held) e0 = __uint_as_float(0x7FC00000u);
      const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
      uint8_t* dst = smem + x * C::kQBytes + trow * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = f32x2_to_f16x2(bf16_lo(w[k]) * e0 * e1, bf16_hi(w[k]) * e0 * e1) ^ sign;
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (128 * 128) + (((c & 7) ^ (trow & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int pos = rq.first + i;
    const int hi = rq.causal ? min(n, pos + 1) : n;           // keys [lo, hi) are seen
    const int lo = kv_first_key(pos, a.window);
    const uint32_t tS = tmem + ((uint32_t)(32 * quad) << 16) + C::kSCol + 128 * x;
    const uint32_t tO = tmem + ((uint32_t)(32 * quad) << 16) + C::kOCol + 128 * x;
    float m = -INFINITY, mf = 0.f, l = 0.f;  // reference of the scores, times f; sum of weights (2^kWeightExp times)
    bool ok = true;
    // page of record ``lane`` of tile j, -1 for none; looked up a tile ahead
    auto page_of = [&](int j) -> int {
      const int key = (t0 + j) * kKeys + 16 * lane;
      return lane < 8 && j < nt && key < n ? table[((SHARED ? rq.base : 0) + key) >> a.cache.page_shift] : -1;
    };
    int next_page = page_of(0);
    if (x < nq) {
      for (int j = 0; j < nt; ++j) {
        const int j0 = (t0 + j) * kKeys;
        // records of this tile that exist: bit k for keys 16 k ..
        const uint32_t have = __ballot_sync(0xffffffffu, next_page >= 0 && next_page < a.cache.num_pages) & 0xFFu;
        next_page = page_of(j + 1);
        if (!mbar_wait_warp(&s_full[x], j & 1, a.status, a.wait.limit_ns, abort_flag)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_after();
        // every row of the warp sees every key of the tile?
        const bool full = __all_sync(0xffffffffu, kv_whole_tile(lo, hi, j0) || !real) && have == 0xFFu;
        if (!full) {  // hidden keys: -inf, put back where the score was
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[16];
            tc_ld16(tS + 16 * c, v);
            tc_ld_wait16(v);
            const bool gone = !((have >> c) & 1u);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int key = j0 + 16 * c + k;
              if (key < lo || key >= hi || gone) v[k] = 0xFF800000u;
            }
            tc_st16(tS + 16 * c, v);
          }
          tc_st_wait();
        }
        // the row's scores, once, in registers
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(tS + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld_wait32(v[c]);
        float mx = -INFINITY;
        {
          float part[4] = {mx, mx, mx, mx};
#pragma unroll
          for (int k = 0; k < 32; k += 2)
#pragma unroll
            for (int c = 0; c < 4; ++c) part[c] = max3(part[c], __uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1]));
          mx = fmaxf(max3(part[0], part[1], part[2]), part[3]);
        }
        // the reference follows the maximum where a weight would pass 2^kSlack
        const bool grow = m == -INFINITY ? mx > -INFINITY : fmaf(mx, f, -mf) > kSlack;
        const bool move = __any_sync(0xffffffffu, grow);
        float al = 1.f;
        if (move && mx > m) {  // (every row of the warp, now that its sums are read anyway)
          const float mf1 = mx * f;
          al = m == -INFINITY ? 0.f : ex2(mf - mf1);
          m = mx;
          mf = mf1;
          l = fabsf(mf1) < kFarScore ? l * al : __uint_as_float(0x7FC00000u);
        }
        {
          const uint64_t f2 = pack2(f, f), off2 = pack2(kWeightExp - mf, kWeightExp - mf);
          uint64_t sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
          if constexpr (FEW) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[16], rest[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float x0, x1;
                unpack2(fma2(pack2(__uint_as_float(v[c][2 * k]), __uint_as_float(v[c][2 * k + 1])), f2, off2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                sum[k & 1] = add2(sum[k & 1], pack2(p0, p1));
                w[k] = prmt(__float_as_uint(p0), __float_as_uint(p1), 0x7632u);  // the upper 8 bits
                rest[k] = f32x2_to_bf16x2(p0 - bf16_lo(w[k]), p1 - bf16_hi(w[k]));
              }
              tc_st16(tS + 16 * c, w);
              tc_st16(tS + 64 + 16 * c, rest);
            }
          } else
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              unpack2(fma2(pack2(__uint_as_float(v[c][2 * k]), __uint_as_float(v[c][2 * k + 1])), f2, off2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              sum[k & 1] = add2(sum[k & 1], pack2(p0, p1));
              w[k] = f32x2_to_f16x2(p0, p1);
            }
            tc_st16(tS + 16 * c, w);
          }
          if (move && j > 0) {
            // O, after the scores, whose registers it takes (the product before
            // these scores is done: one thread's MMAs complete in order)
            if (!mbar_wait_warp(&o_done[x], (j - 1) & 1, a.status, a.wait.limit_ns)) {
              tc_st_wait();
              *abort_flag = 1;
              ok = false;
              break;
            }
            tc_after();
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              uint32_t o[2][32];
              tc_ld32(tO + 64 * c, o[0]);
              tc_ld32(tO + 64 * c + 32, o[1]);
              tc_ld_wait32(o[0]);
              tc_ld_wait32(o[1]);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  uint32_t w[16];
#pragma unroll
                  for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(o[h][16 * q + k]) * al);
                  tc_st16(tO + 64 * c + 32 * h + 16 * q, w);
                }
            }
          }
          tc_st_wait();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
          float l0, l1;
          unpack2(add2(sum[0], sum[1]), l0, l1);
          l += l0 + l1;
        }
      }
      if (ok && nt > 0 && !mbar_wait_warp(&o_done[x], (nt - 1) & 1, a.status, a.wait.limit_ns)) {
        *abort_flag = 1;
        ok = false;
      }
      if (ok) {
        // beyond kFarScore on the way, not held or NaN (a slice of a shared prefix: only for rows whose results are used)
        if (l != l && (!SHARED || r < a.R || (real && kv_row_counts(a, i)))) p.odd[r] = 1;
        __syncwarp();  // (the lookup may part the lanes; loads of tensor memory take them together)
        tc_after();
        if constexpr (SHARED) {
          const size_t to = (size_t)rq.part * a.N * a.Hq + (size_t)(qb + i) * a.Hq + hq;
          // (weights are 2^(S f + (kWeightExp - mf)): that is their reference)
          if (real) a.sh.ml[to] = make_float4(l == 0.f ? -INFINITY : -0.25f * (kWeightExp - mf), l, __int_as_float(127), 0.f);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            if (nt > 0) {
              tc_ld32(tO + 32 * c, v);
              tc_ld_wait32(v);
            }
            if (real && nt > 0) {
              // (32 bytes a store: whole sectors of the row)
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a.sh.o + to * D + 32 * c + k),
                             "r"(v[k]), "r"(v[k + 1]), "r"(v[k + 2]), "r"(v[k + 3]), "r"(v[k + 4]), "r"(v[k + 5]),
                             "r"(v[k + 6]), "r"(v[k + 7])
                             : "memory");
            }
          }
        } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = (size_t)(qb + i) * a.Hq + hq;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (nt > 0) {
            tc_ld32(tO + 32 * c, v);
            tc_ld_wait32(v);
          }
          if (real) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + at * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t o[4] = {0u, 0u, 0u, 0u};
              if (nt > 0 && l != 0.f) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  o[e] = f32x2_to_bf16x2(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
              }
              dst[k] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        if (real && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (mf + lg2(l) - kWeightExp) * 0.6931471805599453f;
        }
      }
    }
  } else if (warp >= kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer of query tile x
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    const int x = warp - kMmaWarp;
    if (nt > 0 && x < nq) {
      constexpr uint32_t id_s = idesc(128, kKeys, false);
      constexpr uint32_t id_o = idesc(128, D, true, FEW);
      const uint64_t dk = sw128(smem_u32(smem), 16), dv = sw128(smem_u32(smem) + C::kVOff, kKeys * 128);
      const uint32_t k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
      const uint32_t qx = (uint32_t)dk + x * (C::kQBytes >> 4), k_lo = (uint32_t)dk + (C::kKOff >> 4), v_lo = (uint32_t)dv;
      const uint32_t ts = tmem + C::kSCol + 128 * x, to = tmem + C::kOCol + 128 * x;
      const int commits = 3 - nq;  // the stages' barriers count one arrival per query tile
      auto scores = [&](int s) {
        const uint32_t ks = k_lo + s * (C::kTile >> 4);
        if (elect_one()) {
          mma_ss_first(ts, desc_at(qx, k_hi, 0), desc_at(ks, k_hi, 0), id_s);
#pragma unroll
          for (int k = 1; k < D / 16; ++k) {
            const uint32_t o = (k >> 2) * (128 * 128) + (k & 3) * 32;
            mma_ss(ts, desc_at(qx, k_hi, o), desc_at(ks, k_hi, o), id_s);
          }
          tc_commit(&s_full[x]);
          for (int c = 0; c < commits; ++c) tc_commit(&k_empty[s]);
        }
        __syncwarp();
      };
      // (every lane waits; a wait that runs out in one lane ends the loop in all)
      auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
      bool ok = all(mbar_wait(q_full, 0, a.status, a.wait.limit_ns) && mbar_wait(&k_full[0], 0, a.status, a.wait.limit_ns));
      tc_after();
      if (ok) scores(0);
      for (int j = 0; j < nt && ok; ++j) {
        const int s = j % S, s1 = (j + 1) % S;
        // (A's turn j comes after B's j - 1, B's after A's j)
        ok = all(mbar_wait(&v_full[s], (j / S) & 1, a.status, a.wait.limit_ns) &&
                 mbar_wait(&p_full[x], j & 1, a.status, a.wait.limit_ns) &&
                 (nq == 1 || (x == 0 && j == 0) || mbar_wait(&turn[x], (j - (x == 0)) & 1, a.status, a.wait.limit_ns)));
        if (!ok) break;
        tc_after();
        const uint32_t vs = v_lo + s * (C::kTile >> 4);
        if (elect_one()) {
          mma_ts_acc(to, ts, desc_at(vs, v_hi, 0), id_o, j > 0);
#pragma unroll
          for (int k = 1; k < kKeys / 16; ++k) mma_ts(to, ts + 8 * k, desc_at(vs, v_hi, k * 16 * 128), id_o);
          if constexpr (FEW) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) mma_ts(to, ts + 64 + 8 * k, desc_at(vs, v_hi, k * 16 * 128), id_o);
          }
          tc_commit(&o_done[x]);
          for (int c = 0; c < commits; ++c) tc_commit(&v_empty[s]);
        }
        __syncwarp();
        if (j + 1 < nt) {
          ok = all(mbar_wait(&k_full[s1], ((j + 1) / S) & 1, a.status, a.wait.limit_ns));
          if (!ok) break;
          tc_after();
          scores(s1);
        }
        if (nq == 2 && lane == 0) mbar_arrive(&turn[1 - x]);
        ok = all(*abort_flag == 0);
      }
      if (!ok) *abort_flag = 1;
      // all issued MMAs complete before tensor memory is released
      if (elect_one()) tc_commit(&drain[x]);
      __syncwarp();
      mbar_wait_warp(&drain[x], 0, a.status, a.wait.limit_ns);
    }
  } else {
    // ---------------------------------------------------------------- converters: one record of a tile per warp
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    const int cw = warp - kConvWarp;
    const int g = lane >> 2, t = lane & 3;
    bool odd = false;
    bool ok = true;
    // codes and scales of a record in registers: lane (g, t) takes two tokens'
    // words of K and four tokens' of V; loaded a tile ahead
    const uint8_t* rec = nullptr;
    int valid = 0;
    uint32_t kc[2][NB], vc[2][NB], ks[2] = {0u, 0u}, vs[4] = {0u, 0u, 0u, 0u};
    auto locate = [&](int j) {
      const int key = (t0 + j) * kKeys + cw * 16;
      rec = nullptr;
      valid = 0;
      if (j < nt && key < n) {
        const int pg = table[((SHARED ? rq.base : 0) + key) >> a.cache.page_shift];
        if (pg >= 0 && pg < a.cache.num_pages) {
          rec = a.cache.data + a.cache.record(pg, kvh, kv_group<SHARED>(a, rq, key));
          valid = min(16, n - key);
        }
      }
    };
    // the scale bytes of token tok (0: past the end, whose values become zeros)
    auto scales = [&](int which, int tok) -> uint32_t {
      if (tok >= valid) return 0u;
      const uint8_t* q = rec + 16 * D + which * (D / 2) + tok * NB;
      return NB == 4 ? *reinterpret_cast<const uint32_t*>(q) : (uint32_t) * reinterpret_cast<const uint16_t*>(q);
    };
    auto words = [&](const uint8_t* q, uint32_t (&c)[NB]) {
      if (NB == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + lane);
        c[0] = x.x; c[1] = x.y; c[NB - 2] = x.z; c[NB - 1] = x.w;
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(q) + lane);
        c[0] = x.x; c[1] = x.y;
      }
    };
    auto load_k = [&]() {
      ks[0] = ks[1] = 0u;
      if (rec) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          words(rec + u * 4 * D, kc[u]);
          ks[u] = scales(0, 8 * u + g);
        }
      }
    };
    auto load_v = [&]() {
      vs[0] = vs[1] = vs[2] = vs[3] = 0u;
      if (rec) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          words(rec + 8 * D + u * 4 * D, vc[u]);
          vs[2 * u] = scales(1, 8 * u + 2 * t);
          vs[2 * u + 1] = scales(1, 8 * u + 2 * t + 1);
        }
      }
    };
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) kc[u][b] = vc[u][b] = 0u;
    locate(0);
    load_k();
    load_v();
    for (int j = 0; j < nt && ok; ++j) {
      const int s = j % S;
      locate(j + 1);
      ok = *abort_flag == 0 && (j < S || mbar_wait(&k_empty[s], ((j / S) - 1) & 1, a.status, a.wait.limit_ns));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int krow = cw * 16 + 8 * u + g;
        uint8_t* dst = smem + C::kKOff + s * C::kTile + krow * 128;
        uint32_t sc[4];
        scale_pairs<NB>(ks[u], sc, odd);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t y[4];
          e2m1x8_to_f16x8(kc[u][b], y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(dst + (b >> 1) * (128 * 128) + ((((b & 1) * 4 + t) ^ (krow & 7)) << 4)) =
              make_uint4(hmul2(y[0], sc[b]), hmul2(y[1], sc[b]), hmul2(y[2], sc[b]), hmul2(y[3], sc[b]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[s]);
      load_k();
      ok = (j < S || mbar_wait(&v_empty[s], ((j / S) - 1) & 1, a.status, a.wait.limit_ns)) && ok;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int w = 0; w < 2; ++w) {  // token 8 u + 2 t + w: dims 4 g .. of every block
          const int krow = cw * 16 + 8 * u + 2 * t + w;
          uint8_t* dst = smem + C::kVOff + s * C::kTile + krow * 128 + 8 * (g & 1);
          uint32_t sc[4];
          scale_pairs<NB>(vs[2 * u + w], sc, odd);
#pragma unroll
          for (int bp = 0; bp < NB / 2; ++bp) {
            uint32_t y[4];
            e2m1x8_to_f16x8(vc[u][w * (NB / 2) + bp], y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              uint2 z = make_uint2(hmul2(y[2 * bb], sc[2 * bp + bb]), hmul2(y[2 * bb + 1], sc[2 * bp + bb]));
              if constexpr (FEW) z = make_uint2(f32x2_to_bf16x2(f16_lo(z.x), f16_hi(z.x)), f32x2_to_bf16x2(f16_lo(z.y), f16_hi(z.y)));
              *reinterpret_cast<uint2*>(dst + bp * (kKeys * 128) + (((bb * 4 + (g >> 1)) ^ (krow & 7)) << 4)) = z;
            }
          }
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[s]);
      load_v();
      // one vote a tile: a lane whose wait ran out goes on to here, so that no lane
      // waits for it above (a vote at each wait: prompt of 8192 tokens 480 us, this
      // 461, lanes leaving one by one, which can hang, 457)
      ok = __all_sync(0xffffffffu, ok) != 0;
    }
    if (!ok) *abort_flag = 1;
    if (odd) p.odd[r] = 1;
  }
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kPromptThreads, 1) kv_prompt_kernel(const PromptParams p) {
  using C = PromptCfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PromptShared<S>& sh = *reinterpret_cast<PromptShared<S>*>(smem + C::kBarOff);
  __shared__ int item[4];  // request, kv head, first row, few keys?
  __shared__ KvRequest request;  // (shared prefix)
  const KvAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int H = a.cache.heads;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.k_full[s], kConvWarps);
      mbar_init(&sh.k_empty[s], 2);
      mbar_init(&sh.v_full[s], kConvWarps);
      mbar_init(&sh.v_empty[s], 2);
    }
    mbar_init(&sh.q_full, kSoftWarps);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.s_full[x], 1);
      mbar_init(&sh.p_full[x], 4 + a.wait.extra_waiters);
      mbar_init(&sh.turn[x], 1);
      mbar_init(&sh.o_done[x], 1);
      mbar_init(&sh.drain[x], 1);
    }
    sh.abort_flag = 0;
    item[0] = -1;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc_alloc(&sh.tmem_slot, C::kCols);
  if (warp == 0) {
    // this CTA's item: the last row tiles of a request first (they see the most keys), heads innermost
    __syncwarp();
    // slices of a shared prefix come first, found without a look at the requests
    const int slices = SHARED ? a.sh.splits * p.slice_tiles * H : 0;
    if (SHARED && (int)blockIdx.x < slices) {
      const int of = blockIdx.x / (p.slice_tiles * H), in = blockIdx.x % (p.slice_tiles * H);
      const KvRequest rq = kv_request<SHARED>(a, a.R + of);
      const long long rows = (long long)rq.ql * p.G, row0 = (long long)(in / H) * 256;
      if (rows > a.sh.row_limit && rows > row0) {
        const int last = (int)((min(row0 + 256, rows) - 1) / p.G);
        const bool few = p.few_rows || rq.n <= kFewKeys || kv_few_rows_among(a, p.G, p.row_limit, (int)(row0 / p.G), last);
        if (lane == 0) {
          item[0] = a.R + of;
          item[1] = in % H;
          item[2] = (int)row0;
          item[3] = few;
          request = rq;
        }
      }
    }
    const long long block = SHARED && (int)blockIdx.x < slices ? -1 : (long long)blockIdx.x - slices;
    long long before = 0;
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const int r = r0 + lane;
      long long rows = 0;
      if (r < a.R) {
        const int qb = min(max(a.query_start[r], 0), a.N);
        rows = (long long)max(min(min(max(a.query_start[r + 1], 0), a.N) - qb, a.max_q_len), 0) * p.G;
      }
      const int tiles = rows > p.row_limit ? (int)((rows + 255) / 256) : 0;
      long long incl = (long long)tiles * H;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const long long off = block - before - (incl - (long long)tiles * H);
      if (off >= 0 && off < (long long)tiles * H) {
        const int qt = tiles - 1 - (int)(off / H);
        item[0] = r;
        item[1] = (int)(off % H);
        item[2] = qt * 256;
        const KvRequest rq = kv_request<SHARED>(a, r);
        const int seen = rq.causal ? min(rq.n, rq.first + item[2] / p.G + 1) : rq.n;
        item[3] = min(seen, a.window ? a.window : seen) <= kFewKeys;
        if (SHARED) request = rq;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
      if (before > block) break;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_slot, 0);
  const int r = item[0];
  if (r >= 0) {
    if constexpr (SHARED) {
      if (item[3]) prompt_item<D, true, true>(p, smem, tmem, r, item[1], item[2], &request);
      else prompt_item<D, false, true>(p, smem, tmem, r, item[1], item[2], &request);
    } else {
      if (item[3]) prompt_item<D, true>(p, smem, tmem, r, item[1], item[2]);
      else prompt_item<D, false>(p, smem, tmem, r, item[1], item[2]);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_after();
    tc_dealloc(tmem, C::kCols);
  }
}

template <int D, bool SHARED>
cudaError_t launch_prompt(const PromptParams& p, unsigned grid, cudaStream_t s) {
  using C = PromptCfg<D>;
  // the register split draws on what the kernel is launched with: never launch it with less
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kv_prompt_kernel<D, SHARED>);
    if (e != cudaSuccess) return e;
    regs.store(attr.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < kLaunchRegs) return cudaErrorInvalidConfiguration;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_shared(kv_prompt_kernel<D, SHARED>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  kv_prompt_kernel<D, SHARED><<<grid, kPromptThreads, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_prompt(const KvAttnArgs& a, int row_limit, int32_t* odd, cudaStream_t s) {
  PromptParams p{};
  p.a = a;
  p.G = a.Hq / a.cache.heads;
  p.row_limit = row_limit;
  p.odd = odd;
  cudaError_t e = cudaMemsetAsync(odd, 0, sizeof(int32_t) * (a.R + a.sh.splits), s);
  if (e != cudaSuccess) return e;
  // at most one tile per 256 rows, and one partial tile per request that has more rows than the limit
  const long long rows = (long long)a.N * p.G;
  const long long most = rows / (row_limit + 1) < a.R ? rows / (row_limit + 1) : a.R;
  long long grid = (rows / 256 + most) * a.cache.heads;
  if (a.sh.splits > 0) {
    // a slice of a shared prefix has all rows (fewer than the limit are streamed)
    p.slice_tiles = rows > a.sh.row_limit ? (int)((rows + 255) / 256) : 0;
    p.few_rows = (long long)a.max_q_len * p.G <= row_limit;
    if (p.few_rows) grid = 0;  // no request of its own has enough rows
    grid += (long long)p.slice_tiles * a.sh.splits * a.cache.heads;
    if (grid == 0) return cudaSuccess;
    return a.cache.D == 128 ? launch_prompt<128, true>(p, (unsigned)grid, s) : launch_prompt<64, true>(p, (unsigned)grid, s);
  }
  if (grid == 0) return cudaSuccess;
  return a.cache.D == 128 ? launch_prompt<128, false>(p, (unsigned)grid, s) : launch_prompt<64, false>(p, (unsigned)grid, s);
}

}  // namespace moe

// The linear layer on MXFP4 weights (linear_a16w4_mxfp4) for many rows: tcgen05 MMAs
// of CTA pairs, weights converted on the way into shared memory.
//
// Measured: 8192 rows x 3584 -> 2 x 3584 gated 234 us, 1,800 TFLOP/s (92 % of the library's
// bf16 matrix product; 265 us on data that draws more power), tensor pipe 76 % active: a
// step's conversions (580 to 690 cycles) are a little longer than its MMAs (512).  250 x 3584 ->
// 8192, K split in two, 22 us: by the slope over K 28 steps of 0.31 us and 13 us beside them (unsplit 10.6): launch, first
// loads and conversion, sums handed over, epilogue.
//
//   D[256 rows of the weight][up to BN tokens] += W[256][16] x[tokens][16]^T
//
// A pair of CTAs (cta_group::2, one SM each) works on a tile: each CTA converts its
// 128 rows of the weight, 64 of K a step, into its shared memory (K-major, 128-byte
// swizzle) and loads one half of the tokens' x by TMA; the first CTA issues the MMAs,
// which read both CTAs' shared memory and leave 128 rows of D in each one's tensor
// memory.  Weights are exact in bf16 with their scale applied, x is bf16 as it
// is, sums are float32.  Rows of the weight are on the M side, so that a tile takes
// any number of tokens (a multiple of 16) and the packed weight, a quarter of its bf16
// size, is what travels: converting it beforehand would write and read it once more.
// SwiGLU: of every 32 rows of a tile, 16 are gate rows and 16 the up rows of the same
// columns, so that one warp holds both.
//
// Warps of a CTA:
//   0 - 7   epilogue: a thread a row of D, two warps sharing its tokens; bias, activation,
//           residual, store
//   8 - 23  converters, in four groups of four warps that take turns: a thread a row of
//           the weight, both blocks of 32 of a step
//   24      MMAs (first CTA)
//   25      TMA of the x tiles
//   26      TMA of the packed weight, four steps (256 of K, a quad) at a time
//   27      scale bytes of a quad to shared memory, loaded a quad ahead of the ring
// Packed weights and scales do not come by loads of the converters: these would have to
// land before the proxy fence that a converter needs each step (a quad took the
// latency of its scale bytes, 1 us), and rows 1,792 bytes apart cost a wavefront of the load unit
// each.
// Two accumulators of 256 columns: the epilogue of one tile runs beside the MMAs of
// the next.  Clusters walk over the tiles, weight tiles innermost.
//
// Where there are fewer tiles than pairs of SMs, K is split (SPLIT): a cluster of 2, 3 or 4
// pairs takes one tile, each pair a run of K; then every CTA hands the other pairs' CTAs
// of the same rows its sums of the tokens (in chunks of 16) that are theirs, in their
// shared memory, and finishes its own.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cooperative_groups.h>

#include "kv_internal.h"
#include "linear.cuh"
#include "tensor_map.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kGroups = 4;              // of converter warps (2: 336 us instead of 327, before the epilogue had 8 warps)
static_assert(kGroups == 4, "a group takes every fourth step of a quad of four");
constexpr int kEpiWarps = 8, kConvWarp = kEpiWarps, kConvWarps = 4 * kGroups;
constexpr int kMmaWarp = kConvWarp + kConvWarps, kTmaWarp = kMmaWarp + 1, kRawWarp = kTmaWarp + 1, kScaleWarp = kRawWarp + 1;
constexpr int kTcThreads = 32 * (kScaleWarp + 1);
constexpr int kRows = 128;              // rows of the weight a CTA
constexpr int kABytes = kRows * 128;    // one step of them in bf16
constexpr int kQuad = 4;                // steps of a load of packed weights
constexpr int kRawStages = 3, kRawBytes = kRows * 128;
constexpr int kScaleBytes = kRows * 8;
constexpr int kChunk = 16;              // tokens that the epilogue takes at a time
constexpr uint32_t kAccCols = 256, kCols = 512;

constexpr int BN = 256;                 // tokens of a tile
constexpr int S = 5;                    // stages of a step
constexpr int kBBytes = BN / 2 * 128, kStage = kABytes + kBBytes;
constexpr int kRawOff = S * kStage, kScaleOff = kRawOff + kRawStages * kRawBytes, kBarOff = kScaleOff + kRawStages * kScaleBytes;
constexpr int kTcSmem = 1024 + kBarOff + 512;
static_assert(kTcSmem <= 227 * 1024, "shared memory");

struct TcShared {
  uint64_t b_full[S];  // this CTA's x tile of a stage
  uint64_t full[S];    // first CTA: weights and x tiles of both
  uint64_t empty[S];   // the stage's MMAs are done
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];  // packed weights of four steps
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_slot;
  volatile int abort_flag;
};

struct LinearTc {
  LinearArgs a;
  int m_tiles, tiles;
  int splits;  // of K, 1 without SPLIT
};

// ------------------------------------------------------------------ pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrives on the barrier at the same place in CTA ``rank`` of the cluster.  What an
// arrival stands for here is shared memory that the MMAs read, or tensor memory: writes
// that a proxy fence or a tcgen05 fence before it has ordered.  It publishes no other writes, so
// it has no release at cluster scope (one such a step, 0.9 us, is what a step took: 604 us instead of 355).
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n mbarrier.arrive.shared::cluster.b64 _, [a];\n}" ::"r"(
          smem_u32(bar)),
      "r"(rank)
      : "memory");
}
// Phase ``parity`` complete?  Sees what arrivals from the other CTA published.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Is it complete now?  (try_wait may suspend the thread while it is not.)
__device__ __forceinline__ bool test_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool test_here(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
// try_wait_cluster by a whole warp, with a limit, one result (see mbar_wait_warp).
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* status, uint64_t limit_ns,
                                             const volatile int* abort) {
  if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
    if ((i & 15u) == 15u && __any_sync(0xffffffffu, *abort != 0)) return false;
    if ((i & 255u) == 255u && __any_sync(0xffffffffu, global_ns() - t0 > limit_ns)) {
      atomicOr(status, kStatusWaitTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void pair_alloc(uint32_t* slot) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(kCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(kCols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on the barriers at this place in both CTAs of the pair (bits of ``mask``) once all MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(mask)
               : "memory");
}
// Four floats to CTA ``rank``'s shared memory.
__device__ __forceinline__ void store_at(float* p, uint32_t rank, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.v4.b32 [a], {%2, %3, %4, %5};\n}" ::"r"(
          smem_u32(p)),
      "r"(rank), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}
// Shared-memory matrix: K-major, 128-byte swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t hi, uint32_t bytes) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
  return d;
}
// kind::f16: bf16 operands, both K-major, float32 sums, M = 256.
__device__ __forceinline__ uint32_t idesc(int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((256u >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The cluster's barrier in two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The weight row of row i (0 .. 127) of CTA ``rank`` in tile mt; -1 outside the weight.
__device__ __forceinline__ int weight_row(const LinearArgs& a, int mt, int rank, int i) {
  if (a.act == LINEAR_ACT_SWIGLU) {
    const int col = mt * 128 + rank * 64 + (i >> 5) * 16 + (i & 15);
    return col < a.cols ? col + (i & 16 ? a.cols : 0) : -1;
  }
  const int row = mt * 256 + rank * 128 + i;
  return row < a.N ? row : -1;
}

// The residuals that ``finish`` adds to a chunk of tokens from ``tok`` on.
__device__ __forceinline__ void fetch_residuals(const LinearArgs& a, int row, int tok, uint16_t (&r)[kChunk]) {
  if (row < 0) return;
  if (a.act == LINEAR_ACT_SWIGLU) {
    const bool up = threadIdx.x & 16;
    uint16_t half[kChunk / 2];
    linear_load_column<kChunk / 2, 2>(a, tok + (up ? 1 : 0), up ? row - a.cols : row, half);
#pragma unroll
    for (int k = 0; k < kChunk / 2; ++k) r[k] = half[k];
  } else {
    linear_load_column<kChunk, 1>(a, tok, row, r);
  }
}
// Bias, activation, residual and store of a weight row's sums for a chunk of tokens from ``tok`` on (the whole warp
// calls it).  ``r``: its residuals, then those of the chunk from ``next`` on (none where that is negative), which are on
// their way while this one is stored and the next one read (loaded where needed, a latency a chunk: 2910 x 64 -> 1084
// 28 us instead of 13, 8192 x 3584 -> 3584 185 instead of 128; without a residual 10 and 117).
template <bool RES>
__device__ __forceinline__ void finish(const LinearArgs& a, int row, float bias, int tok, int next, const uint32_t (&v)[kChunk],
                                       uint16_t (&r)[kChunk]) {
  const int lane = threadIdx.x & 31;
  if (a.act == LINEAR_ACT_SWIGLU) {
    // lanes of gate rows take the even tokens, those of up rows the odd ones
    const bool up = lane & 16;
    float h[kChunk / 2];
#pragma unroll
    for (int k = 0; k < kChunk / 2; ++k) {
      const float x0 = __uint_as_float(v[2 * k]) + bias, x1 = __uint_as_float(v[2 * k + 1]) + bias;
      const float theirs = __shfl_xor_sync(0xffffffffu, up ? x0 : x1, 16);
      h[k] = linear_silu(up ? theirs : x0) * (up ? x1 : theirs);
    }
    if constexpr (RES) {
#pragma unroll
      for (int k = 0; k < kChunk / 2; ++k) h[k] += __uint_as_float((uint32_t)r[k] << 16);
      if (next >= 0) fetch_residuals(a, row, next, r);
    }
    if (row >= 0) linear_store_column<kChunk / 2, 2>(a, tok + (up ? 1 : 0), up ? row - a.cols : row, h);
  } else if (row >= 0) {
    float h[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) h[k] = __uint_as_float(v[k]) + bias;
    if (a.act == LINEAR_ACT_SILU) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) h[k] = linear_silu(h[k]);
    } else if (a.act == LINEAR_ACT_GELU) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) h[k] = linear_act(LINEAR_ACT_GELU, h[k]);
    }
    if constexpr (RES) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) h[k] += __uint_as_float((uint32_t)r[k] << 16);
      if (next >= 0) fetch_residuals(a, row, next, r);
    }
    linear_store_column<kChunk, 1>(a, tok, row, h);
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1) linear_tc_kernel(const __grid_constant__ CUtensorMap map,
                                                                  const __grid_constant__ CUtensorMap wmap, const LinearTc p) {
  extern __shared__ uint8_t smem_raw[];
  // (both CTAs' tiles lie at the same addresses: the launch gives every CTA the same base)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcShared& sh = *reinterpret_cast<TcShared*>(smem + kBarOff);
  const LinearArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // rank within the pair, the pair's first CTA, its run of K
  const int crank = cluster_rank(), rank = crank & 1, first = crank & ~1, z = crank >> 1;
  const int ctas = SPLIT ? 2 * p.splits : 2, cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
  const uint16_t both = (uint16_t)(3u << first);
  const int KB = a.K >> 5;  // blocks of 32
  int q_lo = 0, KS = (KB + 1) >> 1, KQ = (KS + kQuad - 1) / kQuad;  // first quad, steps of 64, quads of steps
  if (SPLIT) {
    const int all = KQ, steps = KS;
    q_lo = all * z / p.splits;
    KQ = all * (z + 1) / p.splits - q_lo;
    KS = min(steps - kQuad * q_lo, kQuad * KQ);
  }
  const uint64_t limit = a.wait.limit_ns;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.b_full[s], 1);
      mbar_init(&sh.full[s], 2 * 4 + a.wait.extra_waiters);  // a group's warps in both CTAs
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&sh.raw_full[s], 2);  // packed weights, scales
      mbar_init(&sh.raw_empty[s], kConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&sh.drain, 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  cluster_arrive();  // warps that touch the other CTA wait for it; copies begin at once
  uint32_t tmem = 0;
  if (warp <= kMmaWarp) {
    if (warp == kMmaWarp) pair_alloc(&sh.tmem_slot);
    tc_before();
    named_bar_sync(1, 32 * (kMmaWarp + 1));
    tc_after();
    tmem = __shfl_sync(0xffffffffu, sh.tmem_slot, 0);
    cluster_wait();  // the other CTA's barriers are there
  }
  // tokens of a tile, and of it what the MMAs take (a multiple of 16)
  auto tokens = [&](int tile, int& t0) -> int {
    t0 = tile / p.m_tiles * BN;
    return min(BN, (min(BN, a.T - t0) + 15) & ~15);
  };

  if (warp < kEpiWarps) {
    // ---------------------------------------------------------------- epilogue: thread = row of D
    const int quad = warp & 3, half = warp >> 2;
    int it = 0;
    for (int tile = cluster; !SPLIT && tile < p.tiles; tile += clusters, ++it) {
      const int buf = it & 1, mt = tile % p.m_tiles;
      int t0;
      const int n = tokens(tile, t0);
      const int row = weight_row(a, mt, rank, 32 * quad + lane);
      const float bias = row >= 0 ? linear_bias(a, row) : 0.f;
      const uint32_t src = tmem + ((uint32_t)(32 * quad) << 16) + kAccCols * buf;
      auto release = [&]() {  // this warp has read its part of the accumulator
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_at(&sh.acc_empty[buf], first);
      };
      auto take = [&](auto res) -> bool {
        constexpr bool RES = decltype(res)::value;
        uint16_t r[kChunk];
        if constexpr (RES) fetch_residuals(a, row, t0 + kChunk * half, r);
        if (!mbar_wait_warp(&sh.acc_full[buf], (it >> 1) & 1, a.status, limit, &sh.abort_flag)) return false;
        tc_after();
        if (kChunk * half >= n) release();
        for (int c = kChunk * half; c < n; c += 2 * kChunk) {
          uint32_t v[kChunk];
          tmem_ld16(src + c, v);
          if (c + 2 * kChunk >= n) release();
          finish<RES>(a, row, bias, t0 + c, c + 2 * kChunk < n ? t0 + c + 2 * kChunk : -1, v, r);
        }
        return true;
      };
      if (!(a.res ? take(std::true_type()) : take(std::false_type()))) {
        sh.abort_flag = 1;
        break;
      }
    }
    // the second CTA: its pair's MMAs are done before its shared and tensor memory go away, too.  (Asked once its tiles have
    // come: from the start on, as by its idle MMA warp, the limit of this wait would be one of the whole call.)
    if (rank == 1 && warp == 0) mbar_wait_warp(&sh.drain, 0, a.status, limit);
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- converters: thread = row of the weight
    const int group = (warp - kConvWarp) >> 2, i = (tid - 32 * kConvWarp) & 127;
    bool ok = true;
    int gs0 = 0, gq = 0;  // steps before this quad, quads
    for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
      for (int quad = 0; quad < KQ && ok; ++quad, ++gq) {
        const int r = gq % kRawStages, steps = min(kQuad, KS - kQuad * quad);
        // (a group takes every fourth step whatever the quads' lengths: the stage of a step of its own has
        // then been left by the step 2 S before, so that the barriers' parities are those of the last two uses.
        // With step ``group`` of each quad, 7 steps lie across the end of a tile whose last quad has 3.)
        const int at = (group - gs0) & (kGroups - 1), gs = gs0 + at, s = gs % S;
        const bool mine = at < steps;
        // (probes now, waits where they failed: the round trips pass beside the conversion.  The x tile is
        // looked for in a free stage only: before, the stage's last x may still be on its way, later than
        // this group's own last one, and the barrier two phases back, where the parity is the same)
        const bool free_now = !mine || gs < S || test_here(&sh.empty[s], ((gs / S) - 1) & 1);
        const bool x_there = !mine || (warp & 3) != 0 || (free_now && test_here(&sh.b_full[s], (gs / S) & 1));
        ok = mbar_wait_warp(&sh.raw_full[r], (gq / kRawStages) & 1, a.status, limit, &sh.abort_flag);
        uint4 w[2][4];
        if (mine) {
          const uint8_t* raw = smem + kRawOff + r * kRawBytes + i * 128;
          const uint32_t sc = *reinterpret_cast<const uint16_t*>(smem + kScaleOff + r * kScaleBytes + i * 8 + 2 * at);
#pragma unroll
          for (int b = 0; b < 2; ++b)
            linear_block(*reinterpret_cast<const uint4*>(raw + (((2 * at + b) ^ (i & 7)) << 4)), (sc >> (8 * b)) & 255u, w[b]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.raw_empty[r]);
        if (mine) {
          if (ok && !__all_sync(0xffffffffu, free_now))
            ok = mbar_wait_warp(&sh.empty[s], ((gs / S) - 1) & 1, a.status, limit, &sh.abort_flag);
          if (!ok) break;
          uint8_t* dst = smem + s * kStage + i * 128;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(dst + (((4 * b + k) ^ (i & 7)) << 4)) = w[b][k];
          fence_proxy_async_smem();
          // one warp of the group answers for the x tile as well
          if ((warp & 3) == 0 && !__all_sync(0xffffffffu, x_there))
            ok = mbar_wait_warp(&sh.b_full[s], (gs / S) & 1, a.status, limit, &sh.abort_flag);
          __syncwarp();
          if (ok && lane == 0) arrive_at(&sh.full[s], first);
        }
        gs0 += steps;
      }
    }
    if (!ok) sh.abort_flag = 1;
  } else if (warp == kTmaWarp) {
    // ---------------------------------------------------------------- x tiles of this CTA's half of the tokens
    if (lane == 0) {
      int gs = 0;
      bool ok = true;
      for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
        int t0;
        const int n = tokens(tile, t0);
        for (int step = 0; step < KS && ok; ++step, ++gs) {
          const int s = gs % S;
          if (gs >= S) ok = sh.abort_flag == 0 && mbar_wait(&sh.empty[s], ((gs / S) - 1) & 1, a.status, limit);
          if (!ok) break;
          mbar_arrive_expect_tx(&sh.b_full[s], kBBytes);
          tma_load_2d(smem + s * kStage + kABytes, &map, 64 * (kQuad * q_lo + step), t0 + rank * (n >> 1), &sh.b_full[s]);
        }
      }
      if (!ok) {
        // copies in flight land before shared memory goes away
        sh.abort_flag = 1;
        for (int k = max(0, gs - S); k < gs; ++k) mbar_wait(&sh.b_full[k % S], (k / S) & 1, a.status, limit);
      }
    }
    __syncwarp();
  } else if (warp == kRawWarp) {
    // ---------------------------------------------------------------- packed weights
    if (lane == 0) {
      int gq = 0;
      bool ok = true;
      for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
        const int mt = tile % p.m_tiles;
        for (int quad = 0; quad < KQ && ok; ++quad, ++gq) {
          const int r = gq % kRawStages;
          if (gq >= kRawStages) ok = sh.abort_flag == 0 && mbar_wait(&sh.raw_empty[r], ((gq / kRawStages) - 1) & 1, a.status, limit);
          if (!ok) break;
          mbar_arrive_expect_tx(&sh.raw_full[r], kRawBytes);
          uint8_t* dst = smem + kRawOff + r * kRawBytes;
          const int at = 128 * (q_lo + quad);
          if (a.act == LINEAR_ACT_SWIGLU) {  // 16 gate rows and the 16 up rows of the same columns a copy
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
              tma_load_3d(dst + k * (32 * 128), &wmap, at, mt * 128 + rank * 64 + 16 * k, 0, &sh.raw_full[r]);
          } else {
            tma_load_3d(dst, &wmap, at, mt * 256 + rank * 128, 0, &sh.raw_full[r]);
          }
        }
      }
      if (!ok) {
        sh.abort_flag = 1;
        for (int k = max(0, gq - kRawStages); k < gq; ++k) mbar_wait(&sh.raw_full[k % kRawStages], (k / kRawStages) & 1, a.status, limit);
      }
    }
    __syncwarp();
  } else if (warp == kScaleWarp) {
    // ---------------------------------------------------------------- scale bytes: four rows a lane
    const bool wide = (((uintptr_t)a.ws | (uintptr_t)KB) & 7) == 0;  // eight bytes lie on such a boundary in every row
    int row[4];
    auto rows_of = [&](int tile) {
#pragma unroll
      for (int k = 0; k < 4; ++k) row[k] = tile < p.tiles ? weight_row(a, tile % p.m_tiles, rank, 32 * k + lane) : -1;
    };
    int ltile = cluster, lquad = 0;
    const int tiles_mine = (p.tiles - cluster + clusters - 1) / clusters;
    rows_of(ltile);
    auto fetch = [&](uint2 (&to)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        to[k] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (row[k] < 0) continue;
        const int b0 = 8 * (q_lo + lquad);
        const uint8_t* src = a.ws + (size_t)row[k] * KB + b0;
        if (wide) {
          to[k] = __ldg(reinterpret_cast<const uint2*>(src));
          continue;
        }
        // three words around the eight bytes, or byte by byte at the ends of the array
        const uintptr_t word = (uintptr_t)src & ~(uintptr_t)3;
        const int n = KB - b0;  // bytes that exist; the others stay 127 (their weights are 0)
        if (word >= (uintptr_t)a.ws && word + 12 <= (uintptr_t)a.ws + (size_t)a.N * KB) {
          const uint32_t* q = reinterpret_cast<const uint32_t*>(word);
          const uint32_t sh = 8u * (uint32_t)((uintptr_t)src & 3), x = __ldg(q), y = __ldg(q + 1), z2 = __ldg(q + 2);
          to[k] = make_uint2(__funnelshift_r(x, y, sh), __funnelshift_r(y, z2, sh));
        } else {
          to[k] = make_uint2(0u, 0u);
#pragma unroll
          for (int b = 0; b < 8; ++b)
            if (b < n) (b < 4 ? to[k].x : to[k].y) |= (uint32_t)__ldg(src + b) << (8 * (b & 3));
        }
        if (n < 8) {
          const uint64_t keep = (1ull << (8 * n)) - 1;
          to[k].x = (to[k].x & (uint32_t)keep) | (0x7F7F7F7Fu & ~(uint32_t)keep);
          to[k].y = (to[k].y & (uint32_t)(keep >> 32)) | (0x7F7F7F7Fu & ~(uint32_t)(keep >> 32));
        }
      }
      if (++lquad == KQ) {
        lquad = 0;
        ltile += clusters;
        rows_of(ltile);
      }
    };
    // quad i's loads go out, then quad i - 1's arrive (two copies of this code: registers of a load
    // on its way cannot be moved)
    const int mine = tiles_mine * KQ;
    bool ok = true;
    auto turn = [&](int i, uint2 (&out)[4], uint2 (&in)[4]) {
      if (i < mine) fetch(out);
      if (i == 0 || i > mine || !ok) return;
      const int gq = i - 1, r = gq % kRawStages;
      if (gq >= kRawStages) ok = mbar_wait_warp(&sh.raw_empty[r], ((gq / kRawStages) - 1) & 1, a.status, limit, &sh.abort_flag);
      if (!ok) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint2*>(smem + kScaleOff + r * kScaleBytes + (32 * k + lane) * 8) = in[k];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.raw_full[r]);
    };
    uint2 u[4], v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = v[k] = make_uint2(0u, 0u);
    for (int i = 0; i <= mine && ok; i += 2) {
      turn(i, u, v);
      turn(i + 1, v, u);
    }
    if (!ok) sh.abort_flag = 1;
  } else if (rank == 0) {
    // ---------------------------------------------------------------- MMAs
    // (the whole warp runs the loop on uniform values, one lane issues)
    const uint64_t da = sw128(smem_u32(smem));
    const uint32_t a_lo = (uint32_t)da, hi = (uint32_t)(da >> 32);
    int s = 0, it = 0;
    uint32_t par = 0;
    bool ok = true, there = false;
    for (int tile = cluster; tile < p.tiles && ok; tile += clusters, ++it) {
      const int buf = it & 1;
      int t0;
      const uint32_t id = idesc(tokens(tile, t0)), d = tmem + kAccCols * buf;
      if (it >= 2) ok = wait_cluster(&sh.acc_empty[buf], ((it >> 1) - 1) & 1, a.status, limit, &sh.abort_flag);
      for (int step = 0; step < KS && ok; ++step) {
        if (!there) ok = wait_cluster(&sh.full[s], par, a.status, limit, &sh.abort_flag);
        if (!ok) break;
        // (the next stage is looked at before this one's MMAs go out: the probe's round trip passes beside them)
        const int s1 = s + 1 == S ? 0 : s + 1;
        const uint32_t par1 = s + 1 == S ? par ^ 1 : par;
        const bool next = test_cluster(&sh.full[s1], par1);
        tc_after();
        const uint32_t lo = a_lo + s * (kStage >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pair_mma(d, desc_at(lo, hi, 32 * k), desc_at(lo, hi, kABytes + 32 * k), id, step > 0 || k > 0);
          pair_commit(&sh.empty[s], both);
          if (step == KS - 1) pair_commit(&sh.acc_full[buf], both);
        }
        __syncwarp();
        s = s1;
        par = par1;
        there = __all_sync(0xffffffffu, next);
      }
    }
    if (!ok) sh.abort_flag = 1;
    // all issued MMAs are done before shared and tensor memory go away
    if (elect_one()) pair_commit(&sh.drain, both);
    __syncwarp();
    mbar_wait_warp(&sh.drain, 0, a.status, limit);
  }
  if (warp > kMmaWarp) cluster_wait();
  tc_before();
  __syncthreads();
  cg::this_cluster().sync();  // no MMA, copy, arrival or read of any CTA's is left
  if constexpr (SPLIT) {
    // chunk c of the tokens is finished by the pair c % splits; kTeams warps take a quarter of the rows
    constexpr int kTeams = (kMmaWarp) / 4;
    const int quad = warp & 3, team = warp >> 2, mt = cluster % p.m_tiles;
    int t0;
    const int chunks = tokens(cluster, t0) / kChunk, most = (chunks + p.splits - 1) / p.splits;
    const uint32_t src = tmem + ((uint32_t)(32 * quad) << 16);
    // sums handed over: [other pair][own chunk][tokens / 4][row 128][token 4]
    float* mine = reinterpret_cast<float*>(smem) + 4 * (32 * quad + lane);
    tc_after();
    if (team < kTeams) {
      for (int c = team; c < chunks; c += kTeams) {
        const int to = c % p.splits;
        if (to == z) continue;
        uint32_t v[kChunk];
        tmem_ld16(src + kChunk * c, v);
        float* dst = mine + (size_t)((z < to ? z : z - 1) * most + c / p.splits) * (kChunk * kRows);
#pragma unroll
        for (int k = 0; k < kChunk; k += 4) store_at(dst + k * kRows, 2 * to + rank, v[k], v[k + 1], v[k + 2], v[k + 3]);
      }
    }
    cg::this_cluster().sync();  // the sums are where they belong
    if (team < kTeams) {
      const int row = weight_row(a, mt, rank, 32 * quad + lane);
      const float bias = row >= 0 ? linear_bias(a, row) : 0.f;
      uint16_t r[kChunk];
      if (a.res) fetch_residuals(a, row, t0 + kChunk * (z + p.splits * team), r);
      for (int c = z + p.splits * team; c < chunks; c += p.splits * kTeams) {
        uint32_t v[kChunk];
        tmem_ld16(src + kChunk * c, v);
        for (int o = 0; o < p.splits - 1; ++o) {
          const float* add = mine + (size_t)(o * most + c / p.splits) * (kChunk * kRows);
#pragma unroll
          for (int k = 0; k < kChunk; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(add + k * kRows);
            v[k] = __float_as_uint(__uint_as_float(v[k]) + x.x);
            v[k + 1] = __float_as_uint(__uint_as_float(v[k + 1]) + x.y);
            v[k + 2] = __float_as_uint(__uint_as_float(v[k + 2]) + x.z);
            v[k + 3] = __float_as_uint(__uint_as_float(v[k + 3]) + x.w);
          }
        }
        const int next = c + p.splits * kTeams;
        if (a.res) finish<true>(a, row, bias, t0 + kChunk * c, next < chunks ? t0 + kChunk * next : -1, v, r);
        else finish<false>(a, row, bias, t0 + kChunk * c, -1, v, r);
      }
    }
    tc_before();
    cg::this_cluster().sync();
  }
  if (warp == kMmaWarp) {
    tc_after();
    pair_dealloc(tmem);
  }
}

int tc_m_tiles(const LinearArgs& a) {
  const int per = a.act == LINEAR_ACT_SWIGLU ? 128 : 256;
  return (a.cols + per - 1) / per;
}

cudaLaunchConfig_t tc_config(int splits, unsigned clusters, cudaLaunchAttribute* attr, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * splits * clusters);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <bool SPLIT>
cudaError_t allow_tc() {
  static std::atomic<unsigned long long> done{0};
  return allow_shared(linear_tc_kernel<SPLIT>, kTcSmem, done);
}

// Clusters of ``splits`` pairs that fit on the current device at once (asked of the runtime once per device).
cudaError_t resident_clusters(int splits, int* n) {
  static std::atomic<int> known[64][5];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* at = dev < 64 ? &known[dev][splits] : nullptr;
  *n = at ? at->load(std::memory_order_relaxed) : 0;
  if (*n > 0) return cudaSuccess;
  if ((e = allow_tc<true>()) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = tc_config(splits, 1, attr, nullptr);
  if ((e = cudaOccupancyMaxActiveClusters(n, linear_tc_kernel<true>, &cfg)) != cudaSuccess) return e;
  if (at) at->store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

template <bool SPLIT>
cudaError_t launch_tc(const LinearArgs& a, int m_tiles, int splits, cudaStream_t s) {
  cudaError_t e = allow_tc<SPLIT>();
  if (e != cudaSuccess) return e;
  CUtensorMap map, wmap;
  if ((e = make_rows_map(&map, a.x, a.T, a.K, a.x_stride, BN / 2, false)) != cudaSuccess) return e;
  const bool gated = a.act == LINEAR_ACT_SWIGLU;
  if ((e = make_bytes_map(&wmap, a.w, gated ? 2 : 1, a.cols, a.K / 2, gated ? 16 : kRows)) != cudaSuccess) return e;
  const LinearTc p{a, m_tiles, m_tiles * ((a.T + BN - 1) / BN), splits};
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = tc_config(splits, (unsigned)(SPLIT ? p.tiles : std::min(p.tiles, a.num_sms / 2)), attr, s);
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<SPLIT>, map, wmap, p);
}

}  // namespace

// Splits of K: as many as leave all clusters resident at once with three quads of K or more
// each (one tile a pair: 250 rows x 3584 -> 8192, 32 tiles, 28.6 us unsplit, 22.3 in 2;
// 64 x 3584 -> 3584, 14 tiles, 24.0 / 17.2 / 15.0 / 14.5 in 1 / 2 / 3 / 4, and
// 128 x 3584 -> 4608, 18 tiles, whose 18 clusters of 8 do not fit at once, 24.9 / 18.3 /
// 17.1 / 29.2; 64 x 512 -> 1024, two quads, 8.8 unsplit and 10.0 in 2).
cudaError_t linear_tc_splits(const LinearArgs& a, int* splits) {
  const long long tiles = (long long)tc_m_tiles(a) * ((a.T + BN - 1) / BN);
  const int quads = (a.K + 255) / 256;
  for (int n = 4; n > 1; --n) {
    if (quads < 3 * n || 2 * n * tiles > a.num_sms) continue;
    int fit = 0;
    const cudaError_t e = resident_clusters(n, &fit);
    if (e != cudaSuccess) return e;
    if (tiles <= fit) {
      *splits = n;
      return cudaSuccess;
    }
  }
  *splits = 1;
  return cudaSuccess;
}

cudaError_t launch_linear_tc(const LinearArgs& a, int splits, cudaStream_t s) {
  return splits > 1 ? launch_tc<true>(a, tc_m_tiles(a), splits, s) : launch_tc<false>(a, tc_m_tiles(a), 1, s);
}

}  // namespace moe

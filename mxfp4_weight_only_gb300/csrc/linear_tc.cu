// The linear layer on MXFP4 weights (linear_a16w4_mxfp4) for many rows: tcgen05 MMAs
// of CTA pairs, weights converted on the way into shared memory.
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
//   24      TMA of the x tiles
//   25      MMAs (first CTA)
//   26      TMA of the packed weight, four steps (256 of K) at a time
// Packed weights come by TMA because loads into registers ahead of their use do not
// outlive the proxy fence that a converter needs each step, and because rows
// 1,792 bytes apart cost a wavefront of the load unit each.
// Two accumulators of 256 columns: the epilogue of one tile runs beside the MMAs of
// the next.  Clusters walk over the tiles, weight tiles innermost.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "kv_internal.h"
#include "linear.cuh"
#include "tensor_map.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kGroups = 4;              // of converter warps
constexpr int kEpiWarps = 8, kConvWarp = kEpiWarps, kConvWarps = 4 * kGroups;
constexpr int kTmaWarp = kConvWarp + kConvWarps, kMmaWarp = kTmaWarp + 1, kRawWarp = kTmaWarp + 2;
constexpr int kTcThreads = 32 * (kRawWarp + 1);
constexpr int kRows = 128;              // rows of the weight a CTA
constexpr int kABytes = kRows * 128;    // one step of them in bf16
constexpr int kQuad = 4;                // steps of a load of packed weights
constexpr int kRawStages = 3, kRawBytes = kRows * 128, kRawRows = 16;
constexpr uint32_t kAccCols = 256, kCols = 512;

template <int BN>
struct TcCfg {
  static constexpr int kStages = BN == 256 ? 5 : BN == 128 ? 7 : 8;
  static constexpr int kBBytes = BN / 2 * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kRawOff = kStages * kStage;
  static constexpr int kBarOff = kRawOff + kRawStages * kRawBytes;
  static constexpr int kSmem = 1024 + kBarOff + 512;
  static_assert(kBBytes % 1024 == 0 && kSmem <= 227 * 1024, "shared memory");
};

template <int S>
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
// it has no release at cluster scope (one such a step, 1 us, is what a step took).
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
// The same by a whole warp, with a limit, one result (see mbar_wait_warp).
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
// Arrives on the barriers at this place in both CTAs of the pair once all MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b16 m;\n mov.b16 m, 3;\n"
      " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(smem_u32(bar))
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
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The weight row of row i (0 .. 127) of CTA ``rank`` in tile mt; -1 outside the weight.
__device__ __forceinline__ int weight_row(const LinearArgs& a, int mt, int rank, int i) {
  if (a.act == LINEAR_ACT_SWIGLU) {
    const int col = mt * 128 + rank * 64 + (i >> 5) * 16 + (i & 15);
    return col < a.cols ? col + (i & 16 ? a.cols : 0) : -1;
  }
  const int row = mt * 256 + rank * 128 + i;
  return row < a.N ? row : -1;
}

template <int BN>
__global__ void __launch_bounds__(kTcThreads, 1) linear_tc_kernel(const __grid_constant__ CUtensorMap map,
                                                                  const __grid_constant__ CUtensorMap wmap, const LinearTc p) {
  using C = TcCfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  // (both CTAs' tiles lie at the same addresses: the launch gives every CTA the same base)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcShared<S>& sh = *reinterpret_cast<TcShared<S>*>(smem + C::kBarOff);
  const LinearArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = cluster_rank(), cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int KB = a.K >> 5, KS = (KB + 1) >> 1, KQ = (KS + kQuad - 1) / kQuad;  // blocks of 32, steps of 64, quads of steps
  const uint64_t limit = a.wait.limit_ns;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sh.b_full[s], 1);
      mbar_init(&sh.full[s], 2 * 4 + a.wait.extra_waiters);  // a group's warps in both CTAs
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&sh.raw_full[s], 1);
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
  cg::this_cluster().sync();  // the other CTA's barriers are there
  if (warp == kMmaWarp) pair_alloc(&sh.tmem_slot);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_slot, 0);
  // tokens of a tile, and of it what the MMAs take (a multiple of 16)
  auto tokens = [&](int tile, int& t0) -> int {
    t0 = tile / p.m_tiles * BN;
    return min(BN, (min(BN, a.T - t0) + 15) & ~15);
  };

  if (warp < kEpiWarps) {
    // ---------------------------------------------------------------- epilogue: thread = row of D
    const int quad = warp & 3, half = warp >> 2;
    const bool gated = a.act == LINEAR_ACT_SWIGLU;
    int it = 0;
    for (int tile = cluster; tile < p.tiles; tile += clusters, ++it) {
      const int buf = it & 1, mt = tile % p.m_tiles;
      int t0;
      const int n = tokens(tile, t0);
      const int row = weight_row(a, mt, rank, 32 * quad + lane);
      const float bias = row >= 0 ? linear_bias(a, row) : 0.f;
      if (!mbar_wait_warp(&sh.acc_full[buf], (it >> 1) & 1, a.status, limit, &sh.abort_flag)) {
        sh.abort_flag = 1;
        break;
      }
      tc_after();
      const uint32_t src = tmem + ((uint32_t)(32 * quad) << 16) + kAccCols * buf;
      auto release = [&]() {  // this warp has read its part of the accumulator
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_at(&sh.acc_empty[buf], 0);
      };
      if (32 * half >= n) release();
      for (int c = 32 * half; c < n; c += 64) {
        uint32_t v[32];
        tmem_ld32(src + c, v);
        if (c + 64 >= n) release();
        if (gated) {
          // lanes of gate rows take the even tokens, those of up rows the odd ones
          const bool up = lane & 16;
          float h[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float x0 = __uint_as_float(v[2 * k]) + bias, x1 = __uint_as_float(v[2 * k + 1]) + bias;
            const float theirs = __shfl_xor_sync(0xffffffffu, up ? x0 : x1, 16);
            h[k] = silu(up ? theirs : x0) * (up ? x1 : theirs);
          }
          if (row >= 0) linear_store_column<16, 2>(a, t0 + c + (up ? 1 : 0), up ? row - a.cols : row, h);
        } else if (row >= 0) {
          float h[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) h[k] = __uint_as_float(v[k]) + bias;
          if (a.act == LINEAR_ACT_SILU) {
#pragma unroll
            for (int k = 0; k < 32; ++k) h[k] = silu(h[k]);
          } else if (a.act == LINEAR_ACT_GELU) {
#pragma unroll
            for (int k = 0; k < 32; ++k) h[k] = linear_act(LINEAR_ACT_GELU, h[k]);
          }
          linear_store_column<32, 1>(a, t0 + c, row, h);
        }
      }
    }
  } else if (warp < kTmaWarp) {
    // ---------------------------------------------------------------- converters: thread = row of the weight
    const int group = (warp - kConvWarp) >> 2, i = (tid - 32 * kConvWarp) & 127;
    auto row_scales = [&](int tile) -> const uint8_t* {
      const int row = tile < p.tiles ? weight_row(a, tile % p.m_tiles, rank, i) : -1;
      return row < 0 ? nullptr : a.ws + (size_t)row * KB;
    };
    const bool wide = (((uintptr_t)a.ws | (uintptr_t)KB) & 1) == 0;
    // The scale bytes of this thread's two blocks of a quad.
    auto scales = [&](const uint8_t* src, int quad) -> uint32_t {
      const int b = 8 * quad + 2 * group;
      if (!src || b >= KB) return 0x7F7Fu;
      src += b;
      if (wide) return __ldg(reinterpret_cast<const uint16_t*>(src));
      return (uint32_t)__ldg(src) | (b + 1 < KB ? (uint32_t)__ldg(src + 1) << 8 : 0x7F00u);
    };
    const uint8_t* here = row_scales(cluster);
    uint32_t sc = scales(here, 0);
    bool ok = true;
    int gs0 = 0, gq = 0;  // steps before this quad, quads
    for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
      const uint8_t* after = row_scales(tile + clusters);
      for (int quad = 0; quad < KQ && ok; ++quad, ++gq) {
        const int r = gq % kRawStages, steps = min(kQuad, KS - kQuad * quad);
        const int gs = gs0 + group, s = gs % S;
        const bool mine = group < steps;
        // (probes now, waits where they failed: the round trips pass beside the conversion)
        const bool free_now = !mine || gs < S || mbar_try_wait(&sh.empty[s], ((gs / S) - 1) & 1);
        const bool x_there = !mine || (warp & 3) != 0 || mbar_try_wait(&sh.b_full[s], (gs / S) & 1);
        ok = mbar_wait_warp(&sh.raw_full[r], (gq / kRawStages) & 1, a.status, limit, &sh.abort_flag);
        uint4 w[2][4];
        if (mine) {
          const uint8_t* raw = smem + C::kRawOff + r * kRawBytes + i * 128;
#pragma unroll
          for (int b = 0; b < 2; ++b)
            linear_block(*reinterpret_cast<const uint4*>(raw + (((2 * group + b) ^ (i & 7)) << 4)), (sc >> (8 * b)) & 255u, w[b]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.raw_empty[r]);
        if (mine) {
          if (ok && !__all_sync(0xffffffffu, free_now))
            ok = mbar_wait_warp(&sh.empty[s], ((gs / S) - 1) & 1, a.status, limit, &sh.abort_flag);
          if (!ok) break;
          uint8_t* dst = smem + s * C::kStage + i * 128;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(dst + (((4 * b + k) ^ (i & 7)) << 4)) = w[b][k];
          fence_proxy_async_smem();
          // one warp of the group answers for the x tile as well
          if ((warp & 3) == 0 && !__all_sync(0xffffffffu, x_there))
            ok = mbar_wait_warp(&sh.b_full[s], (gs / S) & 1, a.status, limit, &sh.abort_flag);
          __syncwarp();
          if (ok && lane == 0) arrive_at(&sh.full[s], 0);
        }
        sc = quad + 1 < KQ ? scales(here, quad + 1) : scales(after, 0);
        gs0 += steps;
      }
      here = after;
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
          mbar_arrive_expect_tx(&sh.b_full[s], C::kBBytes);
          tma_load_2d(smem + s * C::kStage + kABytes, &map, 64 * step, t0 + rank * (n >> 1), &sh.b_full[s]);
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
    // ---------------------------------------------------------------- packed weights, 16 rows a copy
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
#pragma unroll
          for (int k = 0; k < kRows / kRawRows; ++k) {
            const int row = a.act == LINEAR_ACT_SWIGLU ? mt * 128 + rank * 64 + (k >> 1) * 16 + (k & 1) * a.cols
                                                       : mt * 256 + rank * 128 + k * 16;
            tma_load_2d(smem + C::kRawOff + r * kRawBytes + k * kRawRows * 128, &wmap, 128 * quad, row, &sh.raw_full[r]);
          }
        }
      }
      if (!ok) {
        sh.abort_flag = 1;
        for (int k = max(0, gq - kRawStages); k < gq; ++k) mbar_wait(&sh.raw_full[k % kRawStages], (k / kRawStages) & 1, a.status, limit);
      }
    }
    __syncwarp();
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
        tc_after();
        const uint32_t lo = a_lo + s * (C::kStage >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pair_mma(d, desc_at(lo, hi, 32 * k), desc_at(lo, hi, kABytes + 32 * k), id, step > 0 || k > 0);
          pair_commit(&sh.empty[s]);
          if (step == KS - 1) pair_commit(&sh.acc_full[buf]);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          par ^= 1;
        }
        there = __all_sync(0xffffffffu, try_wait_cluster(&sh.full[s], par));
      }
    }
    if (!ok) sh.abort_flag = 1;
    // all issued MMAs are done before shared and tensor memory go away
    if (elect_one()) pair_commit(&sh.drain);
    __syncwarp();
    mbar_wait_warp(&sh.drain, 0, a.status, limit);
  } else {
    mbar_wait_warp(&sh.drain, 0, a.status, limit);
  }
  tc_before();
  __syncthreads();
  cg::this_cluster().sync();  // no MMA, arrival or read of the other CTA's is left
  if (warp == kMmaWarp) {
    tc_after();
    pair_dealloc(tmem);
  }
}

template <int BN>
cudaError_t launch_tc(const LinearArgs& a, int m_tiles, cudaStream_t s) {
  using C = TcCfg<BN>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_shared(linear_tc_kernel<BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = make_rows_map(&map, a.x, a.T, a.K, a.x_stride, BN / 2, false);
  if (e != cudaSuccess) return e;
  CUtensorMap wmap;
  e = make_bytes_map(&wmap, a.w, a.N, a.K / 2, kRawRows);
  if (e != cudaSuccess) return e;
  LinearTc p{a, m_tiles, m_tiles * ((a.T + BN - 1) / BN)};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min(p.tiles, a.num_sms / 2));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_tc_kernel<BN>, map, wmap, p);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearArgs& a, cudaStream_t s) {
  const int per = a.act == LINEAR_ACT_SWIGLU ? 128 : 256;
  const int m_tiles = (a.cols + per - 1) / per, pairs = a.num_sms / 2;
  // tiles of fewer tokens where wide ones would leave SMs without any
  auto tiles = [&](int n) { return (long long)m_tiles * ((a.T + n - 1) / n); };
  if (tiles(256) >= pairs) return launch_tc<256>(a, m_tiles, s);
  if (tiles(128) >= pairs) return launch_tc<128>(a, m_tiles, s);
  return launch_tc<64>(a, m_tiles, s);
}

}  // namespace moe

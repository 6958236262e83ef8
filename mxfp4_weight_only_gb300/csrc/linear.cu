// The linear layer on MXFP4 weights (linear_a16w4_mxfp4) for few rows, or few tiles: the
// weight is streamed from memory, straight into the operands of m16n8k16 MMAs.
//
// Measured (device time in a CUDA graph, weights from memory): 3584 -> 4608, one row
// 5.5 us, 8 rows 5.8, 16 7.5, 24 8.4, 32 9.4; 4096 -> 14336, one row 12.6 us (2.5 TB/s).  Small
// weights: latency of a launch, a load and a reduction; large ones: the issue of the
// exact conversions, five instructions on two weights.
//
//   h[n][token] = sum_k W[n][k] x[token][k]
//
// A CTA takes 16 rows of the weight (SwiGLU: 8 gate rows and the 8 up rows of the
// same columns) and a tile of 8 NT tokens; its 8 warps, and those of the other
// CTAs of its cluster, share K in chunks of 128.  An MMA sums over k in any order
// as long as both operands agree: lane (g, t) = (lane / 4, lane % 4) holds all 32
// values of block t of the chunk, of rows g and g + 8, so it loads its weights in
// two 16-byte words, needs one scale byte a row, and finds the same values of
// token g in 64 bytes of x.  Weights are exact in bf16 with their scale applied,
// x is bf16 as it is, sums are float32.  Partial sums meet in shared memory, those
// of a cluster in its first CTA's.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "kv_internal.h"
#include "linear.cuh"
#include "tensor_map.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kStreamWarps = 8;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes to shared memory, of which ``bytes`` are read (the rest zeros).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Values of x of block b (32 of K) of tokens g, g + 8 ..; zeros past the end of either.
template <int NT>
__device__ __forceinline__ void load_x(const LinearArgs& a, int g, int b, uint4 (&x)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = 8 * n + g;
    const bool there = tok < a.T && 32 * b < a.K;
    const uint4* src = reinterpret_cast<const uint4*>(a.x + (size_t)tok * a.x_stride + 32 * b);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[n][i] = there ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
  }
}
// The products of a chunk: w0, w1 of rows g and g + 8.
template <int NT>
__device__ __forceinline__ void mma_chunk(float (&acc)[NT][4], const uint4 (&w0)[4], const uint4 (&w1)[4], const uint4 (&x)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mma_bf16(acc[n], w0[i].x, w1[i].x, w0[i].y, w1[i].y, x[n][i].x, x[n][i].y);
      mma_bf16(acc[n], w0[i].z, w1[i].z, w0[i].w, w1[i].w, x[n][i].z, x[n][i].w);
    }
}
// A warp's sums of a tile to [token][row].
template <int NT>
__device__ __forceinline__ void store_part(float* part, int g, int t, const float (&acc)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[(8 * n + 2 * t + (k & 1)) * 16 + g + 8 * (k >> 1)] = acc[n][k];
}

// NT: token tiles of 8.  AHEAD: chunks of a warp whose weights are on their way.
template <int NT, int AHEAD>
__global__ void __launch_bounds__(32 * kStreamWarps, 2) linear_stream_kernel(const LinearArgs a) {
  constexpr int COLS = 8 * NT;
  __shared__ float part[kStreamWarps][COLS * 16];
  __shared__ float sum[COLS * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x, splits = gridDim.y, step = kStreamWarps * splits;
  const int KB = a.K >> 5, chunks = (KB + 3) >> 2;
  const bool gated = a.act == LINEAR_ACT_SWIGLU;
  // rows g and g + 8 of the tile
  int row[2];
  bool live[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    row[h] = gated ? tile * 8 + g : tile * 16 + 8 * h + g;
    live[h] = row[h] < a.cols;
    if (gated) row[h] += h * a.cols;
  }
  uint4 wq[AHEAD][2];
  uint32_t sc[AHEAD][2];
  auto load = [&](int p, int c) {
    const int b = 4 * c + t;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      wq[p][h] = make_uint4(0u, 0u, 0u, 0u);
      sc[p][h] = 127u;
      if (live[h] && b < KB) {
        wq[p][h] = load_once(a.w + ((size_t)row[h] * KB + b) * 16);
        sc[p][h] = __ldg(a.ws + (size_t)row[h] * KB + b);
      }
    }
  };
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  const int first = warp * splits + blockIdx.y;
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) load(p, first + p * step);
  for (int c0 = first; c0 < chunks; c0 += AHEAD * step) {
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) {
      const int c = c0 + p * step;
      if (c >= chunks) break;
      uint4 x[NT][4];
      load_x(a, g, 4 * c + t, x);
      uint4 w0[4], w1[4];
      linear_block(wq[p][0], sc[p][0], w0);
      linear_block(wq[p][1], sc[p][1], w1);
      load(p, c + AHEAD * step);
      mma_chunk(acc, w0, w1, x);
    }
  }
  store_part(part[warp], g, t, acc);
  __syncthreads();
  for (int e = threadIdx.x; e < COLS * 16; e += 32 * kStreamWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) v += part[w][e];
    sum[e] = v;
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (splits > 1) {
    cluster.sync();
    if (blockIdx.y == 0) {
      for (int e = threadIdx.x; e < COLS * 16; e += 32 * kStreamWarps) {
        float v = sum[e];
        for (int z = 1; z < splits; ++z) v += *cluster.map_shared_rank(&sum[e], z);
        sum[e] = v;
      }
    }
    cluster.sync();
    if (blockIdx.y) return;
  }
  __syncthreads();
  const int per = gated ? 8 : 16;  // columns of the result a tile
  for (int e = threadIdx.x; e < COLS * per; e += 32 * kStreamWarps) {
    const int n = e / per, r = e % per, col = tile * per + r;
    if (col >= a.cols || n >= a.T) continue;
    float h = sum[n * 16 + r] + linear_bias(a, col);
    if (gated) h = linear_silu(h) * (sum[n * 16 + 8 + r] + linear_bias(a, a.cols + col));
    else h = linear_act(a.act, h);
    linear_store(a, n, col, h);
  }
}

// ------------------------------------------------------------------ many tiles
//
// The same for more tiles than two CTAs an SM hold: resident CTAs walk over them, and a
// warp's next weights are on their way across the end of a tile.  They wait in shared memory,
// each lane's own (cp.async: no registers, so that three CTAs an SM fit), a tile's chunks of a warp filled
// up to a multiple of kWalkAhead.  Measured, one row: 512 -> 28672 7.0 us, with a CTA a tile
// 11.2; 3584 -> 7168 7.3 and 9.2; 4096 -> 14336 12.6 and 14.7; 8192 -> 28672 39.8 and 46.0 (3584 -> 4608,
// two CTAs an SM hold all tiles, 5.7 and 5.5).  16 rows: 8192 -> 28672 70.7 and 75.2.  What bounds it: 4
// instructions a weight, two thirds of the issue slots, ALU pipe 60 %; four chunks ahead are slower.
constexpr int kWalkAhead = 2, kWalkSmem = kStreamWarps * kWalkAhead * 1024;
template <int NT>
constexpr int kWalkCtas = NT == 1 ? 3 : 2;

template <int NT>
__global__ void __launch_bounds__(32 * kStreamWarps, kWalkCtas<NT>) linear_walk_kernel(const LinearArgs a, int tiles) {
  constexpr int COLS = 8 * NT, AHEAD = kWalkAhead;
  __shared__ float part[2][kStreamWarps][COLS * 16];
  extern __shared__ uint4 walk_ring[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;
  const int KB = a.K >> 5, chunks = (KB + 3) >> 2;
  const bool gated = a.act == LINEAR_ACT_SWIGLU;
  const int per = gated ? 8 : 16;  // columns of the result a tile
  constexpr int kRound = AHEAD * kStreamWarps;
  const int end = (chunks + kRound - 1) / kRound * kRound + warp;  // of a warp's chunks warp, warp + 8 ..
  uint4* ring = walk_ring + warp * (AHEAD * 64) + lane;  // [chunk][row g, g + 8][lane]
  uint32_t sc[AHEAD][2];
  // what is loaded next: block t of chunk lc of tile lt, rows g and g + 8 (past the last: another's, not stored)
  int lt = blockIdx.x, lc = warp;
  const uint8_t *wp[2], *sp[2];
  auto point = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = min(gated ? lt * 8 + g : lt * 16 + 8 * h + g, a.cols - 1);
      const size_t at = (size_t)(gated && h ? col + a.cols : col) * KB + 4 * warp + t;
      wp[h] = a.w + at * 16;
      sp[h] = a.ws + at;
    }
  };
  auto load = [&](int p) {
    const bool there = lt < tiles && 4 * lc + t < KB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cp_async16(ring + p * 64 + 32 * h, there ? wp[h] : a.w, there ? 16 : 0);
      sc[p][h] = there ? __ldg(sp[h]) : 127u;
      wp[h] += 64 * kStreamWarps;
      sp[h] += 4 * kStreamWarps;
    }
    cp_async_commit();
    lc += kStreamWarps;
    if (lc == end) {
      lc = warp;
      lt += gridDim.x;
      point();
    }
  };
  point();
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) load(p);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    for (int c0 = warp; c0 < end; c0 += kRound) {
#pragma unroll
      for (int p = 0; p < AHEAD; ++p) {
        const int c = c0 + p * kStreamWarps;
        if (c < chunks) {
          uint4 x[NT][4];
          load_x(a, g, 4 * c + t, x);
          cp_async_wait<AHEAD - 1>();
          uint4 w0[4], w1[4];
          linear_block(ring[p * 64], sc[p][0], w0);
          linear_block(ring[p * 64 + 32], sc[p][1], w1);
          mma_chunk(acc, w0, w1, x);
        }
        load(p);
      }
    }
    store_part(part[buf][warp], g, t, acc);
    __syncthreads();  // (one a tile: the other buffer is written after the next, when all have read this one)
    for (int e = threadIdx.x; e < COLS * per; e += 32 * kStreamWarps) {
      const int n = e / per, r = e % per, col = tile * per + r;
      if (col >= a.cols || n >= a.T) continue;
      float h = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < kStreamWarps; ++w) {
        h += part[buf][w][n * 16 + r];
        if (gated) u += part[buf][w][n * 16 + 8 + r];
      }
      h += linear_bias(a, col);
      if (gated) h = linear_silu(h) * (u + linear_bias(a, a.cols + col));
      else h = linear_act(a.act, h);
      linear_store(a, n, col, h);
    }
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ more than 16 rows
//
// The same products, 32 rows of the weight and up to 32 tokens a CTA, x by TMA: each warp has a ring of its
// own that x of its next kXStages chunks is on its way into, 64 columns a box, zeros
// outside.  (Loads of the lanes, as above, would be 64-byte pieces of eight rows, without
// registers to have the next chunk's under way: 3584 -> 3584, 32 rows 12.1 us instead of
// 9.2, 8192 -> 28672 132 instead of 88.)
constexpr int kXStages = 3;
template <int NT>
constexpr int kXBytes = 8 * NT * 256;  // of a chunk: tokens x 128
template <int NT>
constexpr int kWideSmem = 1024 + kStreamWarps * kXStages * kXBytes<NT>;

template <int NT>
__global__ void __launch_bounds__(32 * kStreamWarps, 1) linear_wide_kernel(const __grid_constant__ CUtensorMap map,
                                                                          const LinearArgs a) {
  constexpr int MT = 2, ROWS = 16 * MT, COLS = 8 * NT, AHEAD = 2, kBytes = kXBytes<NT>;
  static_assert((kStreamWarps + 1) * COLS * ROWS * 4 <= kStreamWarps * kXStages * kBytes, "sums fit into the rings");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bars[kStreamWarps][kXStages];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x, tok0 = blockIdx.z * COLS, splits = gridDim.y, step = kStreamWarps * splits, first = warp * splits + blockIdx.y;
  const int KB = a.K >> 5, chunks = (KB + 3) >> 2, cnt = first < chunks ? (chunks - first + step - 1) / step : 0;
  const bool gated = a.act == LINEAR_ACT_SWIGLU;
  const int per = gated ? ROWS / 2 : ROWS;  // columns of the result a tile
  uint8_t* ring = smem + warp * (kXStages * kBytes);

  auto issue = [&](int i) {  // x of this warp's chunk i: two boxes of 64 columns
    if (lane == 0 && i < cnt) {
      const int s = i % kXStages, k = 128 * (first + i * step);
      mbar_arrive_expect_tx(&bars[warp][s], kBytes);
      tma_load_2d(ring + s * kBytes, &map, k, tok0, &bars[warp][s]);
      tma_load_2d(ring + s * kBytes + kBytes / 2, &map, k + 64, tok0, &bars[warp][s]);
    }
  };
  // weight rows: of row tile m, g and g + 8
  long long row[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = tile * per + (gated ? 8 * m + g : 16 * m + 8 * h + g);
      row[m][h] = col < a.cols ? (long long)(gated && h ? col + a.cols : col) * KB : -1;
    }
  uint4 wq[AHEAD][MT][2];
  uint32_t sc[AHEAD][MT][2];
  auto load = [&](int p, int i) {
    const int b = 4 * (first + i * step) + t;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wq[p][m][h] = make_uint4(0u, 0u, 0u, 0u);
        sc[p][m][h] = 127u;
        if (row[m][h] >= 0 && i < cnt && b < KB) {
          wq[p][m][h] = load_once(a.w + (row[m][h] + b) * 16);
          sc[p][m][h] = __ldg(a.ws + row[m][h] + b);
        }
      }
  };
#pragma unroll
  for (int p = 0; p < AHEAD; ++p) load(p, p);
  if (lane == 0) {
    for (int s = 0; s < kXStages; ++s) mbar_init(&bars[warp][s], 1 + a.wait.extra_waiters);
    fence_barrier_init();
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kXStages; ++i) issue(i);
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;

  bool ok = true;
  int i = 0;
  while (i < cnt && ok) {
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) {
      if (i >= cnt || !ok) break;
      uint4 w[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (lanes of the second box take the block's halves the other way round: the
          // eight reads of x of a quarter warp then fall into different banks)
          const uint4 q = wq[p][m][h];
          linear_block(t & 2 ? make_uint4(q.z, q.w, q.x, q.y) : q, sc[p][m][h], w[m][h]);
        }
      load(p, i + AHEAD);
      const int s = i % kXStages;
      ok = mbar_wait_warp(&bars[warp][s], (i / kXStages) & 1, a.status, a.wait.limit_ns);
      if (!ok) break;
      // block t of the chunk: 16-byte pieces 4 (t & 1) .. of a token's row in box t / 2
      const uint8_t* box = ring + s * kBytes + (t >> 1) * (kBytes / 2);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = *reinterpret_cast<const uint4*>(box + (8 * n + g) * 128 + (((4 * (t & 1) + (k ^ (t & 2))) ^ g) << 4));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma_bf16(acc[m][n], w[m][0][k].x, w[m][1][k].x, w[m][0][k].y, w[m][1][k].y, x[k].x, x[k].y);
            mma_bf16(acc[m][n], w[m][0][k].z, w[m][1][k].z, w[m][0][k].w, w[m][1][k].w, x[k].z, x[k].w);
          }
      }
      __syncwarp();  // the stage has been read
      issue(i + kXStages);
      ++i;
    }
  }
  if (!ok)  // copies in flight land before the ring is used again
    for (int k = i; k < min(i + kXStages, cnt); ++k)
      mbar_wait_warp(&bars[warp][k % kXStages], (k / kXStages) & 1, a.status, a.wait.limit_ns);
  __syncthreads();
  // the warps' sums, in the rings: [warp][token][row]
  float(*part)[COLS * ROWS] = reinterpret_cast<float(*)[COLS * ROWS]>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) part[warp][(8 * n + 2 * t + (k & 1)) * ROWS + 16 * m + g + 8 * (k >> 1)] = acc[m][n][k];
  __syncthreads();
  float* sum = part[kStreamWarps];
  for (int e = threadIdx.x; e < COLS * ROWS; e += 32 * kStreamWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) v += part[w][e];
    sum[e] = v;
  }
  if (splits > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (blockIdx.y == 0)
      for (int e = threadIdx.x; e < COLS * ROWS; e += 32 * kStreamWarps)
        for (int z = 1; z < splits; ++z) sum[e] += *cluster.map_shared_rank(&sum[e], z);
    cluster.sync();
    if (blockIdx.y) return;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < COLS * per; e += 32 * kStreamWarps) {
    const int n = e / per, r = e % per, col = tile * per + r, tok = tok0 + n;
    if (col >= a.cols || tok >= a.T) continue;
    // (gated: of every 16 rows, 8 gates and their ups)
    const int at = n * ROWS + (gated ? 16 * (r >> 3) + (r & 7) : r);
    float h = sum[at] + linear_bias(a, col);
    if (gated) h = linear_silu(h) * (sum[at + 8] + linear_bias(a, a.cols + col));
    else h = linear_act(a.act, h);
    linear_store(a, tok, col, h);
  }
}

// A launch whose CTAs of one tile (gridDim.y of them) form a cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kStreamWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = grid.y;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid.y > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
// K shared between CTAs where there are too few tiles for the SMs, down to one chunk a warp.
// Up to ``limit`` CTAs before the last doubling.
int stream_splits(const LinearArgs& a, int tiles, int limit) {
  int splits = 1;
  while (splits < 8 && tiles * splits < limit && kStreamWarps * splits * 128 < a.K) splits *= 2;
  return splits;
}

int wide_tiles(const LinearArgs& a) {
  const int per = a.act == LINEAR_ACT_SWIGLU ? 16 : 32;
  return (a.cols + per - 1) / per;
}
template <int NT>
cudaError_t launch_wide(const LinearArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_shared(linear_wide_kernel<NT>, kWideSmem<NT>, done);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if ((e = make_rows_map(&map, a.x, a.T, a.K, a.x_stride, 8 * NT, false)) != cudaSuccess) return e;
  const int tiles = wide_tiles(a), tok_tiles = (a.T + 8 * NT - 1) / (8 * NT);
  // (one CTA an SM: no split into a second wave.  112 tiles in two halves 16 us instead of 10)
  const dim3 grid(tiles, stream_splits(a, tiles * tok_tiles, a.num_sms / 2 + 1), tok_tiles);
  return launch_clusters(linear_wide_kernel<NT>, grid, kWideSmem<NT>, s, map, a);
}

template <int NT, int AHEAD>
cudaError_t launch_stream(const LinearArgs& a, cudaStream_t s) {
  const int per = a.act == LINEAR_ACT_SWIGLU ? 8 : 16, tiles = (a.cols + per - 1) / per;
  if (tiles > 2 * a.num_sms)
    return launch_clusters(linear_walk_kernel<NT>, dim3(std::min(tiles, kWalkCtas<NT> * a.num_sms)), kWalkSmem, s, a, tiles);
  return launch_clusters(linear_stream_kernel<NT, AHEAD>, dim3(tiles, stream_splits(a, tiles, a.num_sms)), 0, s, a);
}

}  // namespace

cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t s) {
  // (chunks ahead: what two CTAs an SM have registers for; 8 rows with three CTAs and three
  // chunks 9.5 us instead of 6.2)
  if (a.T <= 8) return launch_stream<1, 4>(a, s);
  if (a.T <= 16) return launch_stream<2, 2>(a, s);
  // 3584 -> 3584: 24 rows 8.2 us, streamed 10.9 (512 -> 512: 3.8 and 2.8); 16 rows 7.5 and 7.6
  // (512 -> 512: 3.4 and 2.4)
  if (a.T <= 24) return launch_wide<3>(a, s);
  return launch_wide<4>(a, s);
}

cudaError_t linear_splits(const LinearArgs& a, int* splits) {
  // 3584 -> 3584: 32 rows 9.2 us, with tcgen05 13.3; more rows take more passes over the weight
  // (in one wave of CTAs: 64 x 3584 -> 2048 9.1 and 13.1, 128 x 8192 -> 1024 15.4 and 19.1, 256 x 512 -> 512
  // 4.4 and 10.2.  In two, of middling depth: 256 x 512 -> 1024 7.8 and 10.2, 1000 x 2048 -> 256 12.0 and 15.2;
  // 96 x 3584 -> 2048 16.6 and 13.6, 64 x 256 -> 4096 7.6 and 6.6.  In three 400 x 1024 -> 1024 12.7 and 12.3.)
  const long long tiles = (long long)wide_tiles(a) * ((a.T + 31) / 32);
  if (a.T <= 32 || tiles <= (a.K >= 512 && a.K <= 2048 ? 2 : 1) * a.num_sms) {
    *splits = 0;
    return cudaSuccess;
  }
  return linear_tc_splits(a, splits);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  int splits = 0;
  const cudaError_t e = linear_splits(a, &splits);
  if (e != cudaSuccess) return e;
  return splits ? launch_linear_tc(a, splits, s) : launch_linear_stream(a, s);
}

}  // namespace moe

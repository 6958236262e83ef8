// The linear layer on MXFP4 weights (linear_a16w4_mxfp4) for few rows: the weight
// is streamed from memory once, straight into the operands of m16n8k16 MMAs.
//
// Measured (device time in a CUDA graph, weights from memory): 3584 -> 4608, one row
// 5.8 us, 8 rows 6.2, 16 7.8, 32 12.4; 4096 -> 14336, one row 15.2 us (1.9 TB/s).  Small
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

#include "linear.cuh"

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

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// NT: token tiles of 8.  AHEAD: chunks of a warp whose weights are on their way.
template <int NT, int AHEAD>
__global__ void __launch_bounds__(32 * kStreamWarps, 2) linear_stream_kernel(const LinearArgs a, int row_tiles) {
  constexpr int COLS = 8 * NT;
  __shared__ float part[kStreamWarps][COLS * 16];
  __shared__ float sum[COLS * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x % row_tiles, tok0 = blockIdx.x / row_tiles * COLS;
  const int splits = gridDim.y, step = kStreamWarps * splits;
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
      const int c = c0 + p * step, b = 4 * c + t;
      if (c >= chunks) break;
      uint4 x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int tok = tok0 + 8 * n + g;
        const bool there = tok < a.T && b < KB;
        const uint4* src = reinterpret_cast<const uint4*>(a.x + (size_t)tok * a.x_stride + 32 * b);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = there ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      }
      uint4 w0[4], w1[4];
      linear_block(wq[p][0], sc[p][0], w0);
      linear_block(wq[p][1], sc[p][1], w1);
      load(p, c + AHEAD * step);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_bf16(acc[n], w0[i].x, w1[i].x, w0[i].y, w1[i].y, x[n][i].x, x[n][i].y);
          mma_bf16(acc[n], w0[i].z, w1[i].z, w0[i].w, w1[i].w, x[n][i].z, x[n][i].w);
        }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][(8 * n + 2 * t + (k & 1)) * 16 + g + 8 * (k >> 1)] = acc[n][k];
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
    const int n = e / per, r = e % per, col = tile * per + r, tok = tok0 + n;
    if (col >= a.cols || tok >= a.T) continue;
    float h = sum[n * 16 + r] + linear_bias(a, col);
    if (gated) h = silu(h) * (sum[n * 16 + 8 + r] + linear_bias(a, a.cols + col));
    else h = linear_act(a.act, h);
    linear_store(a, tok, col, h);
  }
}

template <int NT, int AHEAD>
cudaError_t launch_stream(const LinearArgs& a, cudaStream_t s) {
  const int per = a.act == LINEAR_ACT_SWIGLU ? 8 : 16;
  const int row_tiles = (a.cols + per - 1) / per;
  const long long tiles = (long long)row_tiles * ((a.T + 8 * NT - 1) / (8 * NT));
  // K shared between CTAs where there are too few tiles for the SMs, down to one chunk a warp
  int splits = 1;
  while (splits < 8 && tiles * splits < a.num_sms && kStreamWarps * splits * 128 < a.K) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, splits);
  cfg.blockDim = dim3(32 * kStreamWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = splits;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, linear_stream_kernel<NT, AHEAD>, a, row_tiles);
}

}  // namespace

cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t s) {
  // (chunks ahead: what two CTAs an SM have registers for; 32 rows with one CTA an SM and
  // two chunks ahead 15.8 us instead of 13.7, 8 rows with three CTAs and three chunks 9.5
  // instead of 6.2)
  if (a.T <= 8) return launch_stream<1, 4>(a, s);
  if (a.T <= 16) return launch_stream<2, 2>(a, s);
  return launch_stream<4, 1>(a, s);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  // 3584 -> 3584: 32 rows streamed 12.1 us, on the tensor cores 13.6; 33 rows and more take two
  // passes over the weight if streamed
  if (a.T <= 32) return launch_linear_stream(a, s);
  return launch_linear_tc(a, s);
}

}  // namespace moe

// Internal declarations of the linear layer on MXFP4 weights.
#pragma once

#include "../../include/block_mxfp4.h"
#include "moe_internal.h"
#ifdef __CUDACC__
#include "common.cuh"
#endif

namespace moe {

struct LinearArgs {
  int T, K, N, cols;  // cols: columns of the result
  int act;
  bool f32;           // float32 results
  long long x_stride, res_stride, out_stride;
  const uint16_t* x;
  const uint8_t *w, *ws;
  const uint16_t *bias, *res;
  void* out;
  uint32_t* status;
  int num_sms;
  WaitSettings wait;
};

// Few rows, or few tiles: MMAs from registers (linear.cu).
cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t s);

// Many rows: tensor cores (linear_tc.cu), K split in ``splits``.
cudaError_t linear_tc_splits(const LinearArgs& a, int* splits);
cudaError_t launch_linear_tc(const LinearArgs& a, int splits, cudaStream_t s);

// 0: launch_linear_stream, else the splits of launch_linear_tc.
cudaError_t linear_splits(const LinearArgs& a, int* splits);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);

#ifdef __CUDACC__

// 32 weights of a block as 16 words of two bf16, exact: codes to f16 pairs, each
// value to float32 times 2^(s-127) (a mixed multiply-add), whose upper halves are the bf16
// values, put together by a byte permute.  Scales that f16 does not hold (s = 0: subnormal;
// 255: NaN) are multiplied in bf16 (all so: one row x 3584 -> 4608 5.8 us instead of 5.5, 8192
// rows gated 240 instead of 234).  The ALU pipe, which the conversions and permutes share,
// bounds the tensor-core kernel's converters.
__device__ __forceinline__ void linear_block(const uint4& q, uint32_t s, uint4 (&out)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (s - 103u < 40u) {
    const uint16_t f = s >= 113u ? (s - 112u) << 10 : 1u << (s - 103u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4], o[4];
      e2m1x8_to_f16x8(w[i], h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n fma.rn.f32.f16 %0, l, %3, 0f00000000;\n"
            " fma.rn.f32.f16 %1, h, %3, 0f00000000;\n}"
            : "=f"(lo), "=f"(hi)
            : "r"(h[k]), "h"(f));
        o[k] = prmt(__float_as_uint(lo), __float_as_uint(hi), 0x7632u);
      }
      out[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }
  const uint32_t f = s == 0u ? 0x00400040u : s == 255u ? 0x7FFF7FFFu : s * 0x00800080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4], o[4];
    e2m1x8_to_f16x8(w[i], h[0], h[1], h[2], h[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = bf16x2_mul(prmt(__float_as_uint(f16_lo(h[k])), __float_as_uint(f16_hi(h[k])), 0x7632u), f);
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ float linear_bias(const LinearArgs& a, int row) {
  return a.bias ? __uint_as_float((uint32_t)a.bias[row] << 16) : 0.f;
}

// h (1 + erf(h / sqrt 2)) / 2 = max(h, 0) - |h| q with the normal tail q = e^(-h^2 / 2) t P(t), t = 1 / (1 + 0.34 |h|):
// P, of degree 8, is erfcx(|h| / sqrt 2) / (2 t) to 5.6e-8 of it (at h = 0) for |h| <= 14.5, fitted by reweighted least squares at
// Chebyshev nodes.  2e-7 |h| in all, 3.2e-8 of normal values' root mean square, as with the library's
// normcdff, with which 827 x 160 -> 564 takes 19.3 us instead of 12.2, 1003 x 2080 -> 1111 22.7 instead of 20.6.
__device__ __forceinline__ float gelu(float h) {
  const float a = fabsf(h), t = __fdividef(1.f, fmaf(0.34f, a, 1.f));
  float p = -0.02587643451988697f;
  p = fmaf(p, t, 0.13835705816745758f);
  p = fmaf(p, t, -0.27087101340293884f);
  p = fmaf(p, t, 0.19971758127212524f);
  p = fmaf(p, t, -0.04310628026723862f);
  p = fmaf(p, t, 0.11471360176801682f);
  p = fmaf(p, t, 0.11535170674324036f);
  p = fmaf(p, t, 0.13609223067760468f);
  p = fmaf(p, t, 0.135621577501297f);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * a * -0.72134752044448170f));  // (log2(e) / 2)
  const float q = t * p * e;
  return h > 8.f ? h : fmaf(-a, q, fmaxf(h, 0.f));  // (h > 8: |h| q is below half a step; infinity)
}

// h / (1 + e^-h) by the exponential of -|h|, which neither overflows nor, in CUDA's own expf, loses bits with its
// size (the fast one's argument rounds at |h| 2^-24): 2^-20 of the result, as float32 arithmetic gives.
__device__ __forceinline__ float linear_silu(float h) {
  const float e = expf(-fabsf(h));
  return __fdividef(h > 0.f ? h : h * e, 1.f + e);
}

// The activation of one value (not the gated one).
__device__ __forceinline__ float linear_act(int act, float h) {
  if (act == LINEAR_ACT_SILU) return linear_silu(h);
  if (act == LINEAR_ACT_GELU) return gelu(h);
  return h;
}

// Residual and store of one activated value.
__device__ __forceinline__ void linear_store(const LinearArgs& a, int token, int col, float v) {
  if (a.res) v += __uint_as_float((uint32_t)a.res[(size_t)token * a.res_stride + col] << 16);
  const size_t at = (size_t)token * a.out_stride + col;
  if (a.f32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<uint16_t*>(a.out)[at] = f32_to_bf16_bits(v);
}

// Residuals of column ``col``, of tokens tok, tok + STEP, ..: zeros past the last token.
template <int N, int STEP>
__device__ __forceinline__ void linear_load_column(const LinearArgs& a, int tok, int col, uint16_t (&r)[N]) {
  const int left = (a.T - tok + STEP - 1) / STEP;  // tokens that exist
  const uint16_t* src = a.res + (size_t)tok * a.res_stride + col;
#pragma unroll
  for (int k = 0; k < N; ++k) r[k] = k < left ? src[(size_t)(k * STEP) * a.res_stride] : (uint16_t)0;
}
// Store of N values of column ``col``, of tokens tok, tok + STEP, ..
template <int N, int STEP>
__device__ __forceinline__ void linear_store_column(const LinearArgs& a, int tok, int col, const float (&h)[N]) {
  const int left = (a.T - tok + STEP - 1) / STEP;
  const size_t at = (size_t)tok * a.out_stride + col;
  if (a.f32) {
    float* dst = reinterpret_cast<float*>(a.out) + at;
#pragma unroll
    for (int k = 0; k < N; ++k, dst += STEP * a.out_stride)
      if (k < left) *dst = h[k];
  } else {
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + at;
#pragma unroll
    for (int k = 0; k < N; ++k, dst += STEP * a.out_stride)
      if (k < left) *dst = f32_to_bf16_bits(h[k]);
  }
}

#endif

}  // namespace moe

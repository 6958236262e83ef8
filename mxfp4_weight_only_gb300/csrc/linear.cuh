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

// Few rows: the weight is streamed once (linear.cu).
cudaError_t launch_linear_stream(const LinearArgs& a, cudaStream_t s);

// Many rows: tensor cores (linear_tc.cu).
cudaError_t launch_linear_tc(const LinearArgs& a, cudaStream_t s);

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);

#ifdef __CUDACC__

// 32 weights of a block as 16 words of two bf16, NaN for scale byte 255.
__device__ __forceinline__ void linear_block(const uint4& q, uint32_t s, uint4 (&out)[4]) {
  dequant_block(q, s, out);
  if (s == 255u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
  }
}

__device__ __forceinline__ float linear_bias(const LinearArgs& a, int row) {
  return a.bias ? __uint_as_float((uint32_t)a.bias[row] << 16) : 0.f;
}

// The activation of one value (not the gated one).
__device__ __forceinline__ float linear_act(int act, float h) {
  if (act == LINEAR_ACT_SILU) return silu(h);
  if (act == LINEAR_ACT_GELU) return h * normcdff(h);
  return h;
}

// Residual and store of one activated value.
__device__ __forceinline__ void linear_store(const LinearArgs& a, int token, int col, float v) {
  if (a.res) v += __uint_as_float((uint32_t)a.res[(size_t)token * a.res_stride + col] << 16);
  const size_t at = (size_t)token * a.out_stride + col;
  if (a.f32) reinterpret_cast<float*>(a.out)[at] = v;
  else reinterpret_cast<uint16_t*>(a.out)[at] = f32_to_bf16_bits(v);
}

#endif

}  // namespace moe

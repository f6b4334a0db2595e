// Shared by the kernels of the 8-bit products (w8_linear.cu: few tokens,
// w8_linear_tc.cu: the others).
#pragma once

#include "layer_ops.cuh"

namespace moe_layer {

size_t w8_tc_workspace(int m, int n, int k, int num_sms);
cudaError_t launch_w8_tc(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s);

__device__ __forceinline__ float scale_at(const void* s, int64_t i, int dtype) {
  if (dtype == MOE_LAYER_FP32) return static_cast<const float*>(s)[i];
  const uint32_t w = static_cast<const uint16_t*>(s)[i];
  return dtype == MOE_LAYER_BF16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}
__device__ __forceinline__ void store_y(void* y, int64_t i, float v, int dtype) {
  if (dtype == MOE_LAYER_FP32) static_cast<float*>(y)[i] = v;
  else if (dtype == MOE_LAYER_BF16) static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(y)[i] = __float2half_rn(v);
}

// y of an exact sum, as fp32 has it
__device__ __forceinline__ float scaled(float sum, float w_scale, float x_scale) {
  return __fmul_rn(__fmul_rn(sum, w_scale), x_scale);
}
__device__ __forceinline__ float scaled(int32_t sum, float w_scale, float x_scale) {
  return scaled(__int2float_rn(sum), w_scale, x_scale);
}

}  // namespace moe_layer

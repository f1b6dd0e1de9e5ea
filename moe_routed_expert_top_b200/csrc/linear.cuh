// linear.cuh - the epilogue of the linear product, shared by its few-row and its
// tiled kernels:
//   z = x W^T + bias,  y = act(z) + residual
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace moe {

__device__ __forceinline__ float linear_act(float z, int act) {
  switch (act) {
    case kActRelu:
      return z < 0.0f ? 0.0f : z;  // a NaN stays one
    case kActSilu:
      return z / (1.0f + expf(-z));
    case kActGelu:
      return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    default:
      return z;
  }
}

// d act(z) / dz. silu: s (1 + z (1 - s)), s = 1 / (1 + e^-z); gelu: Phi(z) + z phi(z).
__device__ __forceinline__ float linear_slope(float z, int act) {
  switch (act) {
    case kActRelu:
      return z > 0.0f ? 1.0f : 0.0f;
    case kActSilu: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    case kActGelu:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
             z * expf(-0.5f * z * z) * 0.39894228040143268f;
    default:
      return 1.0f;
  }
}

__device__ __forceinline__ float linear_bias(const LinearEpilogue& e, int n) {
  if (e.bias == nullptr) return 0.0f;
  return e.bias_f32 ? __ldg(static_cast<const float*>(e.bias) + n)
                    : __bfloat162float(static_cast<const __nv_bfloat16*>(e.bias)[n]);
}

// The result of one value, `s` = (x W^T)[m][n], whose bias is `bias` and whose
// residual value is `res`.
__device__ __forceinline__ float linear_result(const LinearEpilogue& e, float s, float bias, float res,
                                               float* z) {
  *z = s + bias;
  return linear_act(*z, e.act) + res;
}

__device__ __forceinline__ float linear_res(const LinearEpilogue& e, long long m, int n) {
  const long long at = m * e.ldr + n;
  return e.res_f32 ? static_cast<const float*>(e.res)[at]
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(e.res)[at]);
}

__device__ __forceinline__ void linear_put(const LinearEpilogue& e, long long m, int n, float y, float z) {
  if (e.z != nullptr) static_cast<__nv_bfloat16*>(e.z)[m * e.ldz + n] = __float2bfloat16(z);
  const long long at = m * e.ldy + n;
  if (e.y_f32)
    static_cast<float*>(e.y)[at] = y;
  else
    static_cast<__nv_bfloat16*>(e.y)[at] = __float2bfloat16(y);
}

__device__ __forceinline__ void linear_store(const LinearEpilogue& e, long long m, int n, float s) {
  float z;
  const float y = linear_result(e, s, linear_bias(e, n), e.res != nullptr ? linear_res(e, m, n) : 0.0f, &z);
  linear_put(e, m, n, y, z);
}

}  // namespace moe

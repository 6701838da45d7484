// values.cuh -- fp32 to and from the types that planes of values are held in; the activations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "product_internal.cuh"

namespace engram {
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float &d, float v) { d = v; }
__device__ __forceinline__ void from_float(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(__half &d, float v) { d = __float2half_rn(v); }

// ENGRAM_ACT_* of one value.
__device__ __forceinline__ float activated(float z, int act) {
  if (act == ENGRAM_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays
  if (act == ENGRAM_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if (act == ENGRAM_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678f));
  return z;
}

}  // namespace
}  // namespace engram

// values.cuh -- fp32 to and from the types that planes of values are held in; the activations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

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

// Sums of squares whose root is right for all finite values: as they are, of the values times 2^-82
// and times 2^80.  Of 2^32 values the second cannot overflow, and the third does not where it serves.
struct Squares {
  float plain, small, large;  // small: of values made small
  __device__ __forceinline__ void add(float v) {
    const float s = v * 0x1p-82f, l = v * 0x1p80f;
    plain = fmaf(v, v, plain), small = fmaf(s, s, small), large = fmaf(l, l, large);
  }
  __device__ __forceinline__ void add(const Squares &o) { plain += o.plain, small += o.small, large += o.large; }
  __device__ __forceinline__ Squares across_lane(int mask) const {
    Squares o{};
    o.plain = __shfl_xor_sync(0xffffffffu, plain, mask);
    o.small = __shfl_xor_sync(0xffffffffu, small, mask);
    o.large = __shfl_xor_sync(0xffffffffu, large, mask);
    return o;
  }
};
// held * v / (|u| + eps) is v * first * second, which overflows and underflows only where the result
// does.  The plain sum serves from 2^-90 (no square that counts beside it was rounded away) up to
// where it overflows.  With a norm and eps of zero zeros stay; with an infinity all become NaN.
struct Norm {
  float first, second;
  __device__ __forceinline__ Norm(const Squares &s, float eps, float held) {
    const float root = s.plain == INFINITY ? s.small : s.plain < 0x1p-90f ? s.large : s.plain;
    first = s.plain == INFINITY ? 0x1p-82f : s.plain < 0x1p-90f ? 0x1p80f : 1.f;
    const float by = sqrtf(root) + eps * first;
    second = by == 0.f ? 0.f : root == INFINITY ? NAN : held / by;
  }
};

}  // namespace
}  // namespace engram

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

// The normal distribution function, with e^(-z^2/2) in `bell`: below zero e^(-w^2/2) G(w), w = -z,
// above it one less that, so that far values keep their bits (1 + erf cancels: 10 % of the value off
// at -5).  G(w) = e^(w^2/2) erfc(w / sqrt 2) / 2 is a polynomial in t = 1 / (1 + 0.31 w) times t, fitted
// for the least relative error on [0, 15]: 1.7e-7, 4.4e-7 with fp32's roundings.
__device__ __forceinline__ float normal_below(float z, float &bell) {
  bell = __expf(-0.5f * z * z);
  const float t = __fdividef(1.f, fmaf(0.31f, fabsf(z), 1.f));
  float g = fmaf(0.0358902439f, t, -0.141817674f);
  g = fmaf(g, t, 0.155456692f);
  g = fmaf(g, t, -0.0152842198f);
  g = fmaf(g, t, 0.110325493f);
  g = fmaf(g, t, 0.107701071f);
  g = fmaf(g, t, 0.12407241f);
  g = fmaf(g, t, 0.123656064f) * t * bell;
  return z < 0.f ? g : 1.f - g;
}

// ENGRAM_ACT_* of one value.
__device__ __forceinline__ float activated(float z, int act) {
  if (act == ENGRAM_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays
  if (act == ENGRAM_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if (act == ENGRAM_ACT_GELU) {
    float bell;
    return z * normal_below(z, bell);
  }
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

// product_grad.cu -- what the product's gradient needs around its two products: the output's
// gradient through the activation, its column sums, and copies of operands whose rows do not
// start on 16 bytes.
//
// act_grad_kernel walks slabs of rows, 8 (or 1, where rows are not aligned) neighbouring columns
// a lane: dz = dy act'(z) is stored as bf16, the operand of the products (rounded once, at most
// 2^-9 of the value), and summed in fp32 before that rounding; a block adds its warps' sums in
// order, a second kernel the slabs', so the result does not depend on timing.  Bound by HBM.
#include <math.h>

#include "launch.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kWarps = 8;

template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T *src, int count, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    alignas(16) T v[8];
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(src);
    } else {
      reinterpret_cast<uint4 *>(v)[0] = reinterpret_cast<const uint4 *>(src)[0];
      reinterpret_cast<uint4 *>(v)[1] = reinterpret_cast<const uint4 *>(src)[1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = i < count ? to_float(src[i]) : 0.f;
  }
}

// dy times the slope of the activation; a unit that relu holds at zero passes nothing on.
__device__ __forceinline__ float through(float dy, float z, int act) {
  if (act == ENGRAM_ACT_RELU) return z > 0.f ? dy : 0.f;
  if (act == ENGRAM_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return dy * (s * (1.f + z * (1.f - s)));
  }
  // gelu: Phi(z) + z phi(z)
  return dy * (0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z));
}

template <int VEC, typename TY, typename TZ>
__global__ void __launch_bounds__(kWarps * 32) act_grad_kernel(const ActGradParams p) {
  dependency_wait();
  __shared__ float sums[kWarps][32 * VEC + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = (int64_t)(blockIdx.x % p.col_blocks) * 32 * VEC + lane * VEC;
  const int64_t slab = blockIdx.x / p.col_blocks;
  const int count = (int)min((int64_t)VEC, p.N - col);
  const int64_t end = min(p.M, (slab + 1) * p.slab_rows);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
  if (count > 0) {
    const TY *dy = static_cast<const TY *>(p.dy) + col;
    const TZ *pre = static_cast<const TZ *>(p.pre) + col;
    __nv_bfloat16 *dz = static_cast<__nv_bfloat16 *>(p.dz) + col;
#pragma unroll 2
    for (int64_t m = slab * p.slab_rows + warp; m < end; m += kWarps) {
      float x[VEC];
      load_vec<VEC>(dy + m * p.dy_stride, count, x);
      if (p.pre) {
        float z[VEC];
        load_vec<VEC>(pre + m * p.pre_stride, count, z);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = through(x[i], z[i], p.act);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] += x[i];
      if (p.dz) {
        if constexpr (VEC == 8) {
          alignas(16) __nv_bfloat16 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) from_float(v[i], x[i]);
          *reinterpret_cast<uint4 *>(dz + m * p.dz_stride) = *reinterpret_cast<const uint4 *>(v);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (i < count) from_float(dz[m * p.dz_stride + i], x[i]);
        }
      }
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) sums[warp][lane * VEC + i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VEC; i += kWarps * 32) {
    const int64_t n = (int64_t)(blockIdx.x % p.col_blocks) * 32 * VEC + i;
    if (n >= p.N) break;
    float s = sums[0][i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += sums[w][i];
    if (p.slabs == 1)
      p.dbias[n] = p.accumulate ? p.dbias[n] + s : s;
    else
      p.partial[slab * p.N + n] = s;
  }
}

// dbias = the slabs' sums, in order.
__global__ void __launch_bounds__(256) join_slabs_kernel(const ActGradParams p) {
  dependency_wait();
  const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= p.N) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.slabs; ++i) s += p.partial[i * p.N + n];
  p.dbias[n] = p.accumulate ? p.dbias[n] + s : s;
}

__global__ void __launch_bounds__(256) pack_kernel(const uint16_t *src, int64_t src_stride, uint16_t *dst,
                                                   int64_t dst_stride, int64_t rows, int64_t cols, int64_t chunks) {
  dependency_wait();
  const int64_t total = rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks, c = (i - r * chunks) * 8;
    alignas(16) uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? src[r * src_stride + c + j] : 0;
    *reinterpret_cast<uint4 *>(dst + r * dst_stride + c) = *reinterpret_cast<const uint4 *>(v);
  }
}

constexpr int kMaxSlabs = 64;

bool vectors(const void *p, int64_t stride, int type) {
  const int64_t step = type == ENGRAM_DTYPE_F32 ? 4 : 8;
  return !p || (((uintptr_t)p & 15) == 0 && stride % step == 0);
}

template <int VEC, typename TY>
cudaError_t launch_typed(const ActGradParams &p, int64_t grid, cudaStream_t stream) {
  if (p.pre_type == ENGRAM_DTYPE_F32)
    return launch(act_grad_kernel<VEC, TY, float>, grid, kWarps * 32, 0, stream, 1, p);
  return launch(act_grad_kernel<VEC, TY, __nv_bfloat16>, grid, kWarps * 32, 0, stream, 1, p);
}

}  // namespace

size_t act_grad_partial_bytes(int64_t M, int64_t N) { return M > 32 ? (size_t)kMaxSlabs * N * sizeof(float) : 0; }

cudaError_t launch_act_grad(ActGradParams p, cudaStream_t stream) {
  const bool wide = p.N % 8 == 0 && vectors(p.dy, p.dy_stride, p.dy_type) && vectors(p.pre, p.pre_stride, p.pre_type) &&
                    vectors(p.dz, p.dz_stride, ENGRAM_DTYPE_BF16);
  const int vec = wide ? 8 : 1;
  p.col_blocks = (int32_t)((p.N + 32 * vec - 1) / (32 * vec));
  // About eight blocks an SM, each of 32 rows at least.
  int64_t slabs = 8 * kSms / p.col_blocks;
  if (slabs > (p.M + 31) / 32) slabs = (p.M + 31) / 32;
  if (slabs > kMaxSlabs) slabs = kMaxSlabs;
  if (slabs < 1) slabs = 1;
  p.slab_rows = (p.M + slabs - 1) / slabs;
  p.slabs = (int32_t)((p.M + p.slab_rows - 1) / p.slab_rows);
  const int64_t grid = (int64_t)p.col_blocks * p.slabs;
  cudaError_t e;
  if (p.dy_type == ENGRAM_DTYPE_F32)
    e = wide ? launch_typed<8, float>(p, grid, stream) : launch_typed<1, float>(p, grid, stream);
  else
    e = wide ? launch_typed<8, __nv_bfloat16>(p, grid, stream) : launch_typed<1, __nv_bfloat16>(p, grid, stream);
  if (e != cudaSuccess || !p.dbias || p.slabs == 1) return e;
  return launch(join_slabs_kernel, (p.N + 255) / 256, 256, 0, stream, 1, p);
}

cudaError_t launch_pack(const void *src, int64_t src_stride, void *dst, int64_t dst_stride, int64_t rows,
                        int64_t cols, cudaStream_t stream) {
  const int64_t chunks = (cols + 7) / 8, blocks = (rows * chunks + 255) / 256;
  return launch(pack_kernel, blocks < 16 * kSms ? blocks : 16 * kSms, 256, 0, stream, 1,
                static_cast<const uint16_t *>(src), src_stride, static_cast<uint16_t *>(dst), dst_stride, rows, cols,
                chunks);
}

}  // namespace engram

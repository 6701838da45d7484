// orthogonalise.cu -- the momentum step of a weight's gradient and the Newton-Schulz iteration
// that replaces the result's singular values by values near one:
//   m = beta m + g,  u = g + beta m (nesterov) or m,  X = u / (|u|_F + eps), then `steps` times
//   A = X X^T (or X^T X, of the shorter side),  B = b A + c A^2,  X = a X + B X (or X B).
//
// Three products a step on the tensor cores (product.cu), two of them symmetric: half of their
// tiles are computed.  The iterate and the two square matrices are held in fp16, times 2^8: all
// their values are bounded (singular values stay under 1.3 with the usual coefficients), so the
// 11 bits of fp16 serve where bf16's 8 cost precision -- against 64 bits the result is 1e-3 to
// 4e-3 off, with bf16 1e-2 to 3e-2 -- at the same rate of the tensor cores.  Times 2^8, values
// down to 2^-22 keep all their bits and singular values up to 255 have room.  The sums of the
// products, the norm and the momentum are fp32.  Bound by the tensor cores for large matrices,
// by the launches for small ones.
#include "launch.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 512;  // blocks a matrix
constexpr float kHeld = 256.f;  // what fp16 values are held times

struct StartDev {
  Plane g, momentum;
  __half *x;
  int64_t x_stride, x_batch;
  float *partial;  // [count][parts]: sums of squares
  int32_t M, N, parts;
  float beta, eps;
  bool nesterov;
};

// u of one element; with `first` the momentum moves.
template <typename T>
__device__ __forceinline__ float update_of(const StartDev &p, int64_t z, int64_t m, int64_t n, bool first) {
  const float g = to_float(static_cast<const T *>(p.g.p)[z * p.g.batch + m * p.g.stride + n]);
  if (!p.momentum.p) return g;
  float *at = static_cast<float *>(p.momentum.p) + z * p.momentum.batch + m * p.momentum.stride + n;
  float v = *at;
  if (first) *at = v = fmaf(p.beta, v, g);
  return p.nesterov ? fmaf(p.beta, v, g) : v;
}

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float sums[kThreads / 32];
  for (int i = 16; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += sums[i];
  return v;
}

// The momentum step and each block's sum of squares of u.
template <typename T>
__global__ void __launch_bounds__(kThreads) momentum_kernel(const StartDev p) {
  dependency_wait();
  const int64_t z = blockIdx.x / p.parts;
  const int part = blockIdx.x - (int)z * p.parts;
  float sum = 0.f;
  for (int m = part; m < p.M; m += p.parts)
    for (int n = threadIdx.x; n < p.N; n += kThreads) {
      const float u = update_of<T>(p, z, m, n, true);
      sum = fmaf(u, u, sum);
    }
  sum = block_sum(sum);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = sum;
}

// X = u / (|u| + eps), held in fp16.
template <typename T>
__global__ void __launch_bounds__(kThreads) normalise_kernel(const StartDev p) {
  dependency_wait();
  const int64_t z = blockIdx.x / p.parts;
  const int part = blockIdx.x - (int)z * p.parts;
  float sum = 0.f;
  for (int i = threadIdx.x; i < p.parts; i += kThreads) sum += p.partial[z * p.parts + i];
  const float by = kHeld / (sqrtf(block_sum(sum)) + p.eps);
  for (int m = part; m < p.M; m += p.parts)
    for (int n = threadIdx.x; n < p.N; n += kThreads)
      p.x[z * p.x_batch + m * p.x_stride + n] = __float2half_rn(update_of<T>(p, z, m, n, false) * by);
}

int64_t padded(int64_t n) { return (n + 63) / 64 * 64; }

struct Layout {
  int64_t x_batch, a_batch;  // elements a matrix
  size_t a, b, x[2], partial, bytes;
};
Layout layout_of(int64_t M, int64_t N, int64_t count) {
  const int64_t r = M < N ? M : N;
  Layout l;
  l.x_batch = M * padded(N);
  l.a_batch = r * padded(r);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.x[0] = take(l.x_batch * count * 2);
  l.x[1] = take(l.x_batch * count * 2);
  l.a = take(l.a_batch * count * 2);
  l.b = take(l.a_batch * count * 2);
  l.partial = take((size_t)kMaxParts * count * sizeof(float));
  l.bytes = at;
  return l;
}

}  // namespace

size_t orthogonalise_workspace_bytes(int64_t M, int64_t N, int64_t count) { return layout_of(M, N, count).bytes; }

cudaError_t launch_orthogonalise(const OrthogonaliseParams &p, void *workspace, cudaStream_t stream) {
  const Layout l = layout_of(p.M, p.N, p.count);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  StartDev s{};
  s.g = p.g;
  s.momentum = p.momentum;
  s.x = reinterpret_cast<__half *>(ws + l.x[0]);
  s.x_stride = padded(p.N);
  s.x_batch = l.x_batch;
  s.partial = reinterpret_cast<float *>(ws + l.partial);
  s.M = (int32_t)p.M;
  s.N = (int32_t)p.N;
  s.beta = p.beta;
  s.eps = p.eps;
  s.nesterov = p.nesterov;
  int64_t parts = (8 * kSms + p.count - 1) / p.count;
  if (parts > p.M) parts = p.M;
  if (parts > kMaxParts) parts = kMaxParts;
  s.parts = (int32_t)parts;
  const bool f32 = p.g.type == ENGRAM_DTYPE_F32;
  cudaError_t e = launch(f32 ? momentum_kernel<float> : momentum_kernel<__nv_bfloat16>, parts * p.count, kThreads, 0,
                         stream, 1, s);
  if (e == cudaSuccess)
    e = launch(f32 ? normalise_kernel<float> : normalise_kernel<__nv_bfloat16>, parts * p.count, kThreads, 0, stream,
               1, s);
  const bool tall = p.M > p.N;
  const int64_t r = tall ? p.N : p.M, w = tall ? p.M : p.N;
  const Plane none{nullptr, 0, 0, ENGRAM_DTYPE_BF16};
  const Plane A{ws + l.a, padded(r), l.a_batch, kTypeF16}, B{ws + l.b, padded(r), l.a_batch, kTypeF16};
  const auto operand = [](const Plane &x, bool t) { return Operand{x.p, x.stride, x.batch, t}; };
  for (int i = 0; i < p.steps && e == cudaSuccess; ++i) {
    const Plane X{ws + l.x[i & 1], padded(p.N), l.x_batch, kTypeF16};
    const bool last = i == p.steps - 1;
    ProductParams q{};
    q.f16 = true;
    q.count = p.count;
    q.status = p.status;
    q.residual = q.pre = none;
    // A, held like X
    q.a = q.b = operand(X, tall);
    q.M = q.N = r;
    q.K = w;
    q.scale = 1.f / kHeld;
    q.out = A;
    q.symmetric = true;
    if ((e = launch_product(q, stream)) != cudaSuccess) break;
    // B
    q.a = q.b = operand(A, false);
    q.K = r;
    q.scale = p.c / kHeld;
    q.residual = A;
    q.residual_scale = p.b;
    q.out = B;
    if ((e = launch_product(q, stream)) != cudaSuccess) break;
    // X
    q.symmetric = false;
    q.a = tall ? operand(X, false) : operand(B, false);
    q.b = tall ? operand(B, false) : operand(X, true);
    q.M = p.M;
    q.N = p.N;
    const float by = last ? p.scale / kHeld : 1.f;
    q.scale = by / kHeld;
    q.residual = X;
    q.residual_scale = p.a * by;
    q.out = last ? p.out : Plane{ws + l.x[(i + 1) & 1], padded(p.N), l.x_batch, kTypeF16};
    e = launch_product(q, stream);
  }
  return e;
}

}  // namespace engram

// orthogonalise.cu -- the momentum step of a weight's gradient and the Newton-Schulz iteration
// that replaces the result's singular values by values near one:
//   m = beta m + g,  u = g + beta m (nesterov) or m,  X = u / (|u|_F + eps), then `steps` times
//   A = X X^T (or X^T X, of the shorter side),  B = b A + c A^2,  X = a X + B X (or X B).
//
// Three products a step on the tensor cores (product.cu), two of them symmetric: half of their
// tiles are computed.  The iterate and the two square matrices are held in fp16, times 2^8: all
// their values are bounded (singular values stay under 1.3 with the usual coefficients), so the
// 11 bits of fp16 serve where bf16's 8 cost precision -- against 64 bits the result is 5e-4 to
// 1e-3 off before its own rounding, with bf16 1e-2 to 3e-2 -- at the same rate of the tensor
// cores.  The square matrices' diagonals, d of A and e of B, stay fp32, and their places in A and B
// are zero:
//   B = (b + c (d_i + d_j)) A + c A^2,   e = b d + c (d^2 + A^2's diagonal),   X = (a + e) X + B X
// (e by X's rows, or its columns where A is X^T X).  Beside many columns A and B are nearly diagonal,
// and a + e is four times as small as e: with e rounded 40 x 3000 is 2.9e-3 off, not 5e-4.  Times
// 2^8, values down to 2^-22 keep all their bits and singular values up to 255 have room.  The sums of
// the products, the norm and the momentum are fp32.  Square matrices whose least singular values nearly
// vanish lose more: their parts of X lie under the roundings of the others, and the iteration brings
// both up; it shows where few singular values make the norm (sides under 16, see the header).  Bound by
// the tensor cores for large matrices (4096 x 6144 of fp32 in 1290 to 1440 us, 1.3 to 1.5 PFLOP/s of the
// products that symmetry leaves, as the power limit lets it), by the launches for small ones (256 x 1536
// in 85 us, 17 launches); 12 of 1024 x 1536 take 450 us, of which the momentum and the norm are 57 (5.2
// TB/s).  A shorter side of at most 128 goes to orthogonalise_small.cu.
#include "launch.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kMostParts = 8 * kSms;  // blocks a matrix
constexpr float kHeld = 256.f;  // what fp16 values are held times

struct StartDev {
  Plane g, momentum;
  __half *x;
  int64_t x_stride, x_batch;
  Squares *partial;  // [count][parts]
  int32_t M, N, parts, lanes;  // lanes: threads a row, a power of two
  float beta, eps;
  bool nesterov;
};

// VEC values of a row; with VEC 4 they are one word of 8 or 16 bytes.
template <int VEC, typename T>
__device__ __forceinline__ void load_values(const T *at, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = to_float(*at);
  } else if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(at);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(at);
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
template <int VEC>
__device__ __forceinline__ void store_values(float *at, const float (&x)[VEC]) {
  if constexpr (VEC == 1)
    *at = x[0];
  else
    *reinterpret_cast<float4 *>(at) = make_float4(x[0], x[1], x[2], x[3]);
}

// f(row, column, u) for a block's share of a matrix in steps of VEC columns, `lanes` threads a row;
// with FIRST the momentum moves.  A thread asks for kAhead steps, then has them.
constexpr int kAhead = 4;
template <int VEC, typename T, bool FIRST, typename F>
__device__ __forceinline__ void over_share(const StartDev &p, int64_t z, int part, F f) {
  const uint32_t lanes = p.lanes, rows = kThreads / lanes, n0 = (threadIdx.x & (lanes - 1)) * VEC;
  const uint32_t M = p.M, N = p.N;
  const T *g = static_cast<const T *>(p.g.p) + z * p.g.batch;
  float *momentum = static_cast<float *>(p.momentum.p) + z * p.momentum.batch;
  uint32_t m = part * rows + threadIdx.x / lanes, n = n0;
  if (n0 >= N) return;
  while (m < M) {
    uint32_t mm[kAhead], nn[kAhead];
    float u[kAhead][VEC], v[kAhead][VEC];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      mm[k] = m, nn[k] = n;
      if (m >= M) continue;
      load_values<VEC>(g + m * p.g.stride + n, u[k]);
      if (p.momentum.p) load_values<VEC>(momentum + m * p.momentum.stride + n, v[k]);
      if ((n += lanes * VEC) >= N) n = n0, m += p.parts * rows;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (mm[k] >= M) continue;
      if (p.momentum.p) {
        if (FIRST) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[k][i] = fmaf(p.beta, v[k][i], u[k][i]);
          store_values<VEC>(momentum + mm[k] * p.momentum.stride + nn[k], v[k]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[k][i] = p.nesterov ? fmaf(p.beta, v[k][i], u[k][i]) : v[k][i];
      }
      f(mm[k], nn[k], u[k]);
    }
  }
}

__device__ __forceinline__ Squares block_sum(Squares v) {
  __shared__ Squares sums[kThreads / 32];
  for (int i = 16; i > 0; i >>= 1) v.add(v.across_lane(i));
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = Squares{};
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v.add(sums[i]);
  return v;
}

// The momentum step and each block's sum of squares of u.
template <int VEC, typename T>
__global__ void __launch_bounds__(kThreads) momentum_kernel(const StartDev p) {
  dependency_wait();
  const int64_t z = blockIdx.x / p.parts;
  const int part = blockIdx.x - (int)z * p.parts;
  Squares sum{};
  over_share<VEC, T, true>(p, z, part, [&](int64_t, int64_t, const float (&u)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum.add(u[i]);
  });
  sum = block_sum(sum);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = sum;
}

// X = u / (|u| + eps), held in fp16.
template <int VEC, typename T>
__global__ void __launch_bounds__(kThreads) normalise_kernel(const StartDev p) {
  dependency_wait();
  const int64_t z = blockIdx.x / p.parts;
  const int part = blockIdx.x - (int)z * p.parts;
  Squares sum{};
  for (int i = threadIdx.x; i < p.parts; i += kThreads) sum.add(p.partial[z * p.parts + i]);
  const Norm norm(block_sum(sum), p.eps, kHeld);
  const auto normal = [&](float v) { return v * norm.first * norm.second; };
  over_share<VEC, T, false>(p, z, part, [&](int64_t m, int64_t n, const float (&u)[VEC]) {
    __half *at = p.x + z * p.x_batch + m * p.x_stride + n;
    if constexpr (VEC == 1) {
      *at = __float2half_rn(normal(u[0]));
    } else {
      __half2 v[2] = {__floats2half2_rn(normal(u[0]), normal(u[1])),
                      __floats2half2_rn(normal(u[2]), normal(u[3]))};
      *reinterpret_cast<uint2 *>(at) = make_uint2(*reinterpret_cast<uint32_t *>(v), *reinterpret_cast<uint32_t *>(v + 1));
    }
  });
}

// Rows of words of four values.
bool words(const Plane &x, int64_t count) {
  const uintptr_t bytes = x.type == ENGRAM_DTYPE_F32 ? 16 : 8;
  return !x.p || (((uintptr_t)x.p & (bytes - 1)) == 0 && x.stride % 4 == 0 && (count == 1 || x.batch % 4 == 0));
}

int64_t padded(int64_t n) { return (n + 63) / 64 * 64; }

struct Layout {
  int64_t x_batch, a_batch;  // elements a matrix
  size_t a, b, x[2], diagonals, partial, bytes;
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
  l.diagonals = take(padded(r) * count * 2 * sizeof(float));
  l.partial = take((size_t)kMostParts * count * sizeof(Squares));
  l.bytes = at;
  return l;
}

}  // namespace

size_t orthogonalise_workspace_bytes(int64_t M, int64_t N, int64_t count) { return layout_of(M, N, count).bytes; }

cudaError_t launch_orthogonalise(const OrthogonaliseParams &p, void *workspace, cudaStream_t stream) {
  if (orthogonalise_small_supported(p)) return launch_orthogonalise_small(p, stream);
  const Layout l = layout_of(p.M, p.N, p.count);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  StartDev s{};
  s.g = p.g;
  s.momentum = p.momentum;
  s.x = reinterpret_cast<__half *>(ws + l.x[0]);
  s.x_stride = padded(p.N);
  s.x_batch = l.x_batch;
  s.partial = reinterpret_cast<Squares *>(ws + l.partial);
  s.M = (int32_t)p.M;
  s.N = (int32_t)p.N;
  s.beta = p.beta;
  s.eps = p.eps;
  s.nesterov = p.nesterov;
  const bool wide = p.N % 4 == 0 && words(p.g, p.count) && words(p.momentum, p.count);
  // As many lanes as a row has values for; of words those of which a row leaves the fewest idle.
  const int64_t vectors = wide ? (p.N + 3) / 4 : p.N;
  const auto taken = [&](int lanes) { return (vectors + lanes - 1) / lanes * lanes; };
  s.lanes = 1;
  for (int lanes = 1; lanes <= kThreads && lanes / 2 < vectors; lanes *= 2)
    if (!wide || lanes <= 32 || taken(lanes) <= taken(s.lanes)) s.lanes = lanes;
  const int64_t rows = kThreads / s.lanes, most = (p.M + rows - 1) / rows;
  const int blocks = (wide ? 4 : 8) * kSms;  // as many as run at once
  int64_t parts = p.count < blocks ? blocks / p.count : 1;
  if (parts > most) parts = most;
  s.parts = (int32_t)parts;
  using Start = void (*)(StartDev);
  static constexpr Start first[4] = {momentum_kernel<1, __nv_bfloat16>, momentum_kernel<1, float>,
                                     momentum_kernel<4, __nv_bfloat16>, momentum_kernel<4, float>};
  static constexpr Start second[4] = {normalise_kernel<1, __nv_bfloat16>, normalise_kernel<1, float>,
                                      normalise_kernel<4, __nv_bfloat16>, normalise_kernel<4, float>};
  const int which = 2 * wide + (p.g.type == ENGRAM_DTYPE_F32);
  cudaError_t e = launch(first[which], parts * p.count, kThreads, 0, stream, 1, s);
  if (e == cudaSuccess) e = launch(second[which], parts * p.count, kThreads, 0, stream, 1, s);
  const bool tall = p.M > p.N;
  const int64_t r = tall ? p.N : p.M, w = tall ? p.M : p.N;
  const Plane none{nullptr, 0, 0, ENGRAM_DTYPE_BF16};
  const Plane A{ws + l.a, padded(r), l.a_batch, kTypeF16}, B{ws + l.b, padded(r), l.a_batch, kTypeF16};
  float *const of_a = reinterpret_cast<float *>(ws + l.diagonals), *const of_b = of_a + padded(r) * p.count;
  const auto operand = [](const Plane &x, bool t) { return Operand{x.p, x.stride, x.batch, t}; };
  for (int i = 0; i < p.steps && e == cudaSuccess; ++i) {
    const Plane X{ws + l.x[i & 1], padded(p.N), l.x_batch, kTypeF16};
    const bool last = i == p.steps - 1;
    ProductParams q{};
    q.f16 = q.newton = true;
    q.diag_batch = padded(r);
    q.diag_scale = 1.f / kHeld;
    q.count = p.count;
    q.status = p.status;
    q.residual = q.pre = none;
    // A, held like X
    q.a = q.b = operand(X, tall);
    q.M = q.N = r;
    q.K = w;
    q.scale = 1.f / kHeld;
    q.out = A;
    q.diag_out = of_a;
    q.symmetric = true;
    if ((e = launch_product(q, stream)) != cudaSuccess) break;
    // B
    q.a = q.b = operand(A, false);
    q.K = r;
    q.scale = p.c / kHeld;
    q.residual = A;
    q.residual_scale = p.b;
    q.out = B;
    q.diag_in = of_a;
    q.diag_out = of_b;
    q.diag_rows = q.diag_columns = true;
    q.diag_by = p.c;
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
    q.diag_in = of_b;
    q.diag_out = nullptr;
    q.diag_rows = !tall;
    q.diag_columns = tall;
    q.diag_by = by;
    q.out = last ? p.out : Plane{ws + l.x[(i + 1) & 1], padded(p.N), l.x_batch, kTypeF16};
    e = launch_product(q, stream);
  }
  return e;
}

}  // namespace engram

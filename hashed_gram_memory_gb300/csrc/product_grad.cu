// product_grad.cu -- what the product's gradient needs around its two products: the output's
// gradient through the activation, its column sums, and copies of operands whose rows do not
// start on 16 bytes.
//
// act_grad_kernel walks slabs of rows, 8 (or 1, where rows are not aligned) neighbouring columns
// a thread: dz = dy act'(z) is stored as bf16, the operand of the products (at most 2^-8 of the value
// off), for fp32 outputs with a second matrix of what that rounding left (the two are at most 2^-16
// off), and summed in fp32 before any rounding; a block adds its rows' sums in
// order, of more than 1024 rows a second kernel the slabs', so the result does not depend on timing.
// Bound by HBM: 16,411 x 2573 of fp32 dy and pre take 69 us, 6.1 TB/s, with 8 rows of single columns
// ahead of a thread and 4 blocks an SM (4 rows and 5 blocks: 104).
#include <math.h>

#include <type_traits>

#include "launch.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256, kMostThreads = 1024;

template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T *src, int count, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    alignas(16) T v[8];
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(v) = __ldg(reinterpret_cast<const uint4 *>(src));
    } else {
      reinterpret_cast<uint4 *>(v)[0] = __ldg(reinterpret_cast<const uint4 *>(src));
      reinterpret_cast<uint4 *>(v)[1] = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = i < count ? to_float(__ldg(src + i)) : 0.f;
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
  float bell;
  const float below = normal_below(z, bell);
  return dy * fmaf(z * 0.39894228f, bell, below);
}

// What a rounding left; nothing of a value that is not finite, or that only its rounding is not.
__device__ __forceinline__ float left_over(float x, __nv_bfloat16 rounded) {
  const float r = to_float(rounded);
  return fabsf(r) < INFINITY ? x - r : 0.f;
}

// DEEP rows, `step` apart, of a thread's VEC columns: all loads, then the others.  REST: dz_rest is
// written too, `rest` elements behind dz (asked at run time it took 512 x 4096 1.5 us longer).
template <int VEC, int DEEP, bool REST, typename TY, typename TZ>
__device__ __forceinline__ void some_rows(const ActGradParams &p, const TY *dy, const TZ *pre, __nv_bfloat16 *dz,
                                          int64_t rest, int64_t step, int count, float (&sum)[VEC]) {
  constexpr bool kAct = !std::is_same_v<TZ, void>;
  float x[DEEP][VEC], z[DEEP][VEC];
#pragma unroll
  for (int d = 0; d < DEEP; ++d) {
    load_vec<VEC>(dy + d * step * p.dy_stride, count, x[d]);
    if constexpr (kAct) load_vec<VEC>(pre + d * step * p.pre_stride, count, z[d]);
  }
#pragma unroll
  for (int d = 0; d < DEEP; ++d) {
    if constexpr (kAct) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[d][i] = through(x[d][i], z[d][i], p.act);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] += x[d][i];
    if (p.dz) {
      __nv_bfloat16 *to = dz + d * step * p.dz_stride;
      if constexpr (VEC == 8) {
        alignas(16) __nv_bfloat16 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) from_float(v[i], x[d][i]);
        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(v);
        if constexpr (REST) {
#pragma unroll
          for (int i = 0; i < 8; ++i) from_float(v[i], left_over(x[d][i], v[i]));
          *reinterpret_cast<uint4 *>(to + rest) = *reinterpret_cast<const uint4 *>(v);
        }
      } else {
        from_float(*to, x[d][0]);
        if constexpr (REST) {
          __nv_bfloat16 v;
          from_float(v, x[d][0]);
          from_float(to[rest], left_over(x[d][0], v));
        }
      }
    }
  }
}

// A block has `lanes` threads a row, VEC columns each.  TZ void: no activation.
template <int VEC, int THREADS, bool REST, typename TY, typename TZ>
__global__ void __launch_bounds__(THREADS) act_grad_kernel(const ActGradParams p) {
  dependency_wait();
  __shared__ float sums[THREADS * VEC];
  const int lanes = p.lanes, rows = THREADS / lanes, row = threadIdx.x / lanes, at = threadIdx.x & (lanes - 1);
  const int64_t col0 = (int64_t)(blockIdx.x % p.col_blocks) * lanes * VEC, col = col0 + at * VEC;
  const int64_t slab = blockIdx.x / p.col_blocks;
  const int count = (int)min((int64_t)VEC, p.N - col);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
  if (count > 0) {
    constexpr int kDeep = VEC == 1 ? 8 : 2;
    const int64_t m = slab * p.slab_rows + row, end = min(p.M, (slab + 1) * p.slab_rows);
    int left = m < end ? (int)((end - 1 - m) / rows + 1) : 0;
    const TY *dy = static_cast<const TY *>(p.dy) + m * p.dy_stride + col;
    const TZ *pre = nullptr;
    if constexpr (!std::is_same_v<TZ, void>) pre = static_cast<const TZ *>(p.pre) + m * p.pre_stride + col;
    __nv_bfloat16 *dz = static_cast<__nv_bfloat16 *>(p.dz) + m * p.dz_stride + col;
    const int64_t rest = REST ? static_cast<__nv_bfloat16 *>(p.dz_rest) - static_cast<__nv_bfloat16 *>(p.dz) : 0;
    const auto move = [&](int n) {
      dy += n * rows * p.dy_stride;
      if constexpr (!std::is_same_v<TZ, void>) pre += n * rows * p.pre_stride;
      dz += n * rows * p.dz_stride;
      left -= n;
    };
    for (; left >= kDeep; move(kDeep)) some_rows<VEC, kDeep, REST, TY, TZ>(p, dy, pre, dz, rest, rows, count, sum);
#pragma unroll 1
    for (; left > 0; move(1)) some_rows<VEC, 1, REST, TY, TZ>(p, dy, pre, dz, rest, rows, count, sum);
  }
  if (!p.dbias) return;
  // sums[row][column of the block]
#pragma unroll
  for (int i = 0; i < VEC; ++i) sums[(row * lanes + at) * VEC + i] = sum[i];
  __syncthreads();
  // First the rows in a few groups, then those.
  const int columns = lanes * VEC, groups = columns < THREADS ? THREADS / columns : 1;
  if (groups > 1) {
    const int i = threadIdx.x % columns, share = rows / groups, r0 = threadIdx.x / columns * share;
    float s = sums[r0 * columns + i];
    for (int r = 1; r < share; ++r) s += sums[(r0 + r) * columns + i];
    sums[r0 * columns + i] = s;
    __syncthreads();
  }
  const int step = rows / groups;
  for (int i = threadIdx.x; i < columns && col0 + i < p.N; i += THREADS) {
    float s = sums[i];
    for (int r = groups > 1 ? step : 1; r < rows; r += groups > 1 ? step : 1) s += sums[r * columns + i];
    const int64_t n = col0 + i;
    if (p.slabs == 1)
      p.dbias[n] = p.accumulate ? p.dbias[n] + s : s;
    else
      p.partial[slab * p.N + n] = s;
  }
}

// dbias = the slabs' sums: a block has 32 columns, its warps some slabs each, in order.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) join_slabs_kernel(const ActGradParams p) {
  dependency_wait();
  __shared__ float sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  const int begin = p.slabs * warp / kJoinWarps, end = p.slabs * (warp + 1) / kJoinWarps;
  float s = 0.f;
  if (n < p.N) {
#pragma unroll 8
    for (int i = begin; i < end; ++i) s += p.partial[i * p.N + n];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || n >= p.N) return;
  for (int i = 1; i < kJoinWarps; ++i) s += sums[i][lane];
  p.dbias[n] = p.accumulate ? p.dbias[n] + s : s;
}

// Copies rows of 16-bit values to rows on 16 bytes, zeros up to the next 8.  A lane two neighbouring
// columns, so that a warp reads and stores whole lines; kPackRows rows of them at a time: all loads,
// then the stores.  A row that does not start on 4 bytes is read in words all the same, of which a lane
// shifts its two values together; at the first and last rows, where such words would reach beyond
// the matrix, values are read one by one.  16,411 x 1278 and 2573 x 1278 together: 23 us; 37,056 x 576
// with odd strides 21 us, 4.1 TB/s (52 with values one by one: the instructions are what counts).
constexpr int kPackRows = 8;
__global__ void __launch_bounds__(256) pack_kernel(const PackParams p) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  for (int k = 0; k < p.count; ++k) {
    const Packed &part = p.part[k];
    const int cols = (int)part.cols, padded = (cols + 7) / 8 * 8, pieces = (padded / 2 + 31) / 32;
    const int64_t total = (part.rows + kPackRows - 1) / kPackRows * pieces;
    const int64_t end = (part.rows - 1) * part.src_stride + cols;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
      int64_t group;  // a 64-bit division takes longer than the copy
      if (total <= UINT32_MAX)
        group = (uint32_t)i / (uint32_t)pieces;
      else
        group = i / pieces;
      const int c0 = (int)(i - group * pieces) * 64, c = c0 + lane * 2;
      const int64_t r0 = group * kPackRows;
      const uint16_t *src = part.src + r0 * part.src_stride + c;
      uint16_t *dst = part.dst + r0 * part.dst_stride + c;
      // A lane's words end at most 66 columns on from c0: inside the row, or in those behind it.
      if ((r0 > 0 || c0 > 0) && r0 + kPackRows <= part.rows &&
          (r0 + kPackRows - 1) * part.src_stride + c0 + 66 <= end) {
        uint32_t low[kPackRows], high[kPackRows];
#pragma unroll
        for (int j = 0; j < kPackRows; ++j) {
          const uintptr_t at = reinterpret_cast<uintptr_t>(src + j * part.src_stride);
          const uint32_t *word = reinterpret_cast<const uint32_t *>(at & ~(uintptr_t)3);
          low[j] = __ldg(word);
          high[j] = at & 2 ? __ldg(word + 1) : 0;
        }
        const uint32_t keep = c + 1 < cols ? ~0u : c < cols ? 0xffffu : 0u;
        if (c < padded) {
#pragma unroll
          for (int j = 0; j < kPackRows; ++j) {
            const uint32_t shift = reinterpret_cast<uintptr_t>(src + j * part.src_stride) & 2 ? 16 : 0;
            *reinterpret_cast<uint32_t *>(dst + j * part.dst_stride) = __funnelshift_r(low[j], high[j], shift) & keep;
          }
        }
      } else if (c < padded) {
        const int rows = (int)min((int64_t)kPackRows, part.rows - r0);
        uint32_t v[kPackRows];
#pragma unroll
        for (int j = 0; j < kPackRows; ++j)
          if (j < rows) {
            const uint32_t lo = c < cols ? __ldg(src + j * part.src_stride) : 0;
            const uint32_t hi = c + 1 < cols ? __ldg(src + j * part.src_stride + 1) : 0;
            v[j] = lo | hi << 16;
          }
#pragma unroll
        for (int j = 0; j < kPackRows; ++j)
          if (j < rows) *reinterpret_cast<uint32_t *>(dst + j * part.dst_stride) = v[j];
      }
    }
  }
}

constexpr int kMaxSlabs = 64;
constexpr int64_t kOneSlab = 1024;  // up to so many rows a block takes them all, and nothing is joined

bool vectors(const void *p, int64_t stride, int type) {
  const int64_t step = type == ENGRAM_DTYPE_F32 ? 4 : 8;
  return !p || (((uintptr_t)p & 15) == 0 && stride % step == 0);
}

template <int VEC, bool REST, typename TY, typename TZ>
cudaError_t launch_threads(const ActGradParams &p, int64_t grid, cudaStream_t stream) {
  if (p.threads == kThreads)
    return launch(act_grad_kernel<VEC, kThreads, REST, TY, TZ>, grid, kThreads, 0, stream, 1, p);
  return launch(act_grad_kernel<VEC, kMostThreads, REST, TY, TZ>, grid, kMostThreads, 0, stream, 1, p);
}
template <int VEC, bool REST, typename TY>
cudaError_t launch_typed(const ActGradParams &p, int64_t grid, cudaStream_t stream) {
  if (!p.pre) {
    // A bf16 dy by itself leaves nothing to a second matrix.
    if constexpr (REST && std::is_same_v<TY, __nv_bfloat16>)
      return cudaErrorInvalidValue;
    else
      return launch_threads<VEC, REST, TY, void>(p, grid, stream);
  }
  if (p.pre_type == ENGRAM_DTYPE_F32) return launch_threads<VEC, REST, TY, float>(p, grid, stream);
  return launch_threads<VEC, REST, TY, __nv_bfloat16>(p, grid, stream);
}
template <int VEC, typename TY>
cudaError_t launch_rest(const ActGradParams &p, int64_t grid, cudaStream_t stream) {
  return p.dz_rest ? launch_typed<VEC, true, TY>(p, grid, stream) : launch_typed<VEC, false, TY>(p, grid, stream);
}

}  // namespace

size_t act_grad_partial_bytes(int64_t M, int64_t N) {
  return M > kOneSlab ? (size_t)kMaxSlabs * N * sizeof(float) : 0;
}

cudaError_t launch_act_grad(ActGradParams p, cudaStream_t stream) {
  const bool wide = p.N % 8 == 0 && vectors(p.dy, p.dy_stride, p.dy_type) && vectors(p.pre, p.pre_stride, p.pre_type) &&
                    vectors(p.dz, p.dz_stride, ENGRAM_DTYPE_BF16);
  const int vec = wide ? 8 : 1;
  // As many blocks as run at once, each of 32 rows at least; of few rows, blocks of fewer columns.
  int64_t slabs = 1;
  p.lanes = 32;
  p.threads = kThreads;
  const auto blocks = [&] { return (p.N + p.lanes * vec - 1) / (p.lanes * vec); };
  if (p.M > kOneSlab) {
    slabs = 4 * kSms / blocks();
    if (slabs > (p.M + 31) / 32) slabs = (p.M + 31) / 32;
    if (slabs > kMaxSlabs) slabs = kMaxSlabs;
    if (slabs < 1) slabs = 1;
  } else {
    const int least = vec == 8 ? 4 : 16;
    if (p.M > kThreads / 8) p.threads = kMostThreads;
    while (p.lanes > least && p.threads / p.lanes < p.M && blocks() < kSms) p.lanes /= 2;
  }
  p.col_blocks = (int32_t)blocks();
  p.slab_rows = (p.M + slabs - 1) / slabs;
  p.slabs = (int32_t)((p.M + p.slab_rows - 1) / p.slab_rows);
  const int64_t grid = (int64_t)p.col_blocks * p.slabs;
  cudaError_t e;
  if (p.dy_type == ENGRAM_DTYPE_F32)
    e = wide ? launch_rest<8, float>(p, grid, stream) : launch_rest<1, float>(p, grid, stream);
  else
    e = wide ? launch_rest<8, __nv_bfloat16>(p, grid, stream) : launch_rest<1, __nv_bfloat16>(p, grid, stream);
  if (e != cudaSuccess || !p.dbias || p.slabs == 1) return e;
  return launch(join_slabs_kernel, (p.N + 31) / 32, 32 * kJoinWarps, 0, stream, 1, p);
}

cudaError_t launch_pack(const PackParams &p, cudaStream_t stream) {
  int64_t blocks = 1;
  for (int i = 0; i < p.count; ++i) {
    const Packed &part = p.part[i];
    const int64_t warps = (part.rows + kPackRows - 1) / kPackRows * (((part.cols + 7) / 8 * 4 + 31) / 32);
    if ((warps + 7) / 8 > blocks) blocks = (warps + 7) / 8;
  }
  return launch(pack_kernel, blocks < 8 * kSms ? blocks : 8 * kSms, 256, 0, stream, 1, p);
}

}  // namespace engram

// product_few.cu -- the product for up to 16 rows of a, as decode steps of a few slots have them.
//
// Reading b is the work (2 bytes for 2 M operations), and what counts beside it is how soon the
// first bytes are asked for and how little comes after the last: no tensor memory to allocate, no
// descriptors to fetch, no CTAs to join.  So a warp loads its operands from memory straight into
// the registers of mma.sync (m16n8k16): 16 rows of b against 8 (or twice 8) rows of a.  The order of
// K inside an instruction is free as long as both operands agree, so a lane's part is 8 neighbouring
// values of a row, one 16-byte word, for every two instructions.  Those words come through shared
// memory, copied asynchronously kDeep steps ahead, and each lane reads back what it copied itself:
// nothing to wait for but its own copies.  A block has 16 rows of b, its warps take 32 of K in turn
// and add their sums in shared memory, always in the same order.  1 x 4096 x 6144 takes 12.0 us, 50 MB
// of b at 4.2 TB/s, about 4 us of them before the first and after the last bytes.
#include <atomic>

#include "launch.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kRows = 16;  // of b a block
constexpr int kWarps = 8;  // of a block at most
constexpr int kSegment = 48;  // steps that the instructions' sums run on: 768 values in each

struct FewDev {
  const uint16_t *a, *b;
  int64_t a_stride, b_stride, K;
  Plane out, residual, pre;
  const void *bias;
  int32_t M, N, bias_type, act, warps;
  float scale, residual_scale;
};

__device__ __forceinline__ float load_one(const void *p, int64_t at, int type) {
  return type == ENGRAM_DTYPE_F32 ? static_cast<const float *>(p)[at]
                                  : to_float(static_cast<const __nv_bfloat16 *>(p)[at]);
}
__device__ __forceinline__ void store_one(void *p, int64_t at, int type, float v) {
  if (type == ENGRAM_DTYPE_F32)
    static_cast<float *>(p)[at] = v;
  else
    from_float(static_cast<__nv_bfloat16 *>(p)[at], v);
}

// Copies the 8 values of a row from k on into shared memory; zeros past K.
__device__ __forceinline__ void copy8(uint32_t dst, const uint16_t *row, int64_t k, int64_t K, bool has) {
  const int64_t left = has && k < K ? 2 * (K - k) : 0;
  const uint32_t bytes = left >= 16 ? 16 : left > 0 ? (uint32_t)left : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(bytes ? row + k : row), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 read16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// c (16 x 8) += a (16 x 16) b (16 x 8).
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// EIGHTS: times 8 rows of a.
template <int EIGHTS>
struct Ring {
  static constexpr int kDeep = EIGHTS == 1 ? 8 : 6;
  static constexpr uint32_t kStep = (2 + EIGHTS) * 512, kBytes = kDeep * kStep;  // of a warp
};

// SEGMENTS: the instructions' sums are added up in fp32 registers every kSegment steps.
template <int EIGHTS, bool SEGMENTS>
__global__ void __launch_bounds__(kWarps * 32) few_rows_kernel(const __grid_constant__ FewDev p) {
  using R = Ring<EIGHTS>;
  constexpr int kColumns = 8 * EIGHTS;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ float sums[kWarps][kRows][kColumns + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = p.warps;
  const int n0 = blockIdx.x * kRows, g = lane >> 2, t = lane & 3;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(sm) + warp * R::kBytes + lane * 16;
  const uint16_t *b0 = p.b + (int64_t)(n0 + g) * p.b_stride, *b1 = b0 + 8 * p.b_stride, *a = p.a + g * p.a_stride;
  const bool has0 = n0 + g < p.N, has1 = n0 + g + 8 < p.N;
  // Two steps share a 128-byte line of a row.
  const int64_t first = warp * 64 + t * 8, step = warps * 64;
  const int steps = p.K > warp * 64 ? 2 * (int)((p.K + step - 1 - warp * 64) / step) : 0;
  dependency_wait();
  const auto copy = [&](int i) {
    if (i < steps) {
      const uint32_t at = mine + (i % R::kDeep) * R::kStep;
      const int64_t k = first + (i >> 1) * step + (i & 1) * 32;
      copy8(at, has0 ? b0 : p.b, k, p.K, has0);
      copy8(at + 512, has1 ? b1 : p.b, k, p.K, has1);
#pragma unroll
      for (int e = 0; e < EIGHTS; ++e) {
        const bool has = e * 8 + g < p.M;
        copy8(at + (2 + e) * 512, has ? a + e * 8 * p.a_stride : p.a, k, p.K, has);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Two sums each, as the instruction's own do not round to nearest: 8192 long 1e-6 off in one.
  float acc[EIGHTS][2][4];
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[e][i / 4][i % 4] = 0.f;
  [[maybe_unused]] float total[EIGHTS][4] = {};
  [[maybe_unused]] int left = kSegment;
  for (int i = 0; i < R::kDeep - 1; ++i) copy(i);
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kDeep - 2) : "memory");
    const uint32_t at = mine + (i % R::kDeep) * R::kStep;
    const uint4 w0 = read16(at), w1 = read16(at + 512);
    uint4 v[EIGHTS];
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) v[e] = read16(at + (2 + e) * 512);
    copy(i + R::kDeep - 1);
#pragma unroll
    for (int e = 0; e < EIGHTS; ++e) {
      mma(acc[e][0], w0.x, w1.x, w0.y, w1.y, v[e].x, v[e].y);
      mma(acc[e][1], w0.z, w1.z, w0.w, w1.w, v[e].z, v[e].w);
    }
    if constexpr (SEGMENTS) {
      if (--left == 0) {
        left = kSegment;
#pragma unroll
        for (int e = 0; e < EIGHTS; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            total[e][j] += acc[e][0][j] + acc[e][1][j];
            acc[e][0][j] = acc[e][1][j] = 0.f;
          }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < EIGHTS; ++e) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[e][0][j] += acc[e][1][j];
      if constexpr (SEGMENTS) acc[e][0][j] += total[e][j];
    }
    sums[warp][g][e * 8 + 2 * t] = acc[e][0][0];
    sums[warp][g][e * 8 + 2 * t + 1] = acc[e][0][1];
    sums[warp][g + 8][e * 8 + 2 * t] = acc[e][0][2];
    sums[warp][g + 8][e * 8 + 2 * t + 1] = acc[e][0][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kColumns; i += warps * 32) {
    const int r = i % kRows, m = i / kRows, n = n0 + r;
    if (m >= p.M || n >= p.N) continue;
    float z = sums[0][r][m];
    for (int w = 1; w < warps; ++w) z += sums[w][r][m];
    z *= p.scale;
    if (p.bias) z += load_one(p.bias, n, p.bias_type);
    if (p.pre.p) store_one(p.pre.p, m * p.pre.stride + n, p.pre.type, z);
    z = activated(z, p.act);
    if (p.residual.p)
      z = fmaf(p.residual_scale, load_one(p.residual.p, m * p.residual.stride + n, p.residual.type), z);
    store_one(p.out.p, m * p.out.stride + n, p.out.type, z);
  }
}

// More than 48 KB of shared memory have to be allowed, once a device.
template <int EIGHTS, bool SEGMENTS>
cudaError_t launch_eights(const FewDev &d, int64_t grid, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(few_rows_kernel<EIGHTS, SEGMENTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWarps * Ring<EIGHTS>::kBytes);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  return launch(few_rows_kernel<EIGHTS, SEGMENTS>, grid, d.warps * 32, d.warps * Ring<EIGHTS>::kBytes, stream, 1, d);
}

}  // namespace

bool few_rows_supported(const ProductParams &p) {
  // Up to 8 rows always: 8 x 4096 x 6144 12.4 us and 13.4 by clusters, 1 x 4096 x 6144 12.0 and 13.1,
  // 8 x 8192 x 8192 27.5 and 28.9.  From 9 rows on that every block reads all rows of a costs more than it
  // saves where b is large, with the shape: 16 x 2048 x 4096 6.2 and 8.0; 16 x 4096 x 6144 14.4 and 13.4,
  // 16 x 4096 x 5120 12.4 and 11.9, 16 x 1024 x 16,384 19.0 and 12.8, but 16 x 4096 x 4096 9.8 and 10.8.
  return (p.M <= 8 || (p.M <= 16 && p.N * p.K <= 12 << 20)) && p.count == 1 && !p.symmetric && !p.f16 && !p.a_two && !p.a.t &&
         !p.b.t && p.out.type != kTypeF16;
}

cudaError_t launch_few_rows(const ProductParams &p, cudaStream_t stream) {
  FewDev d{};
  d.a = static_cast<const uint16_t *>(p.a.p);
  d.b = static_cast<const uint16_t *>(p.b.p);
  d.a_stride = p.M > 1 ? p.a.stride : 0;
  d.b_stride = p.N > 1 ? p.b.stride : 0;
  d.K = p.K;
  d.out = p.out;
  d.residual = p.residual;
  d.pre = p.pre;
  d.bias = p.bias;
  d.bias_type = p.bias_type;
  d.M = (int32_t)p.M;
  d.N = (int32_t)p.N;
  d.act = p.act;
  d.scale = p.scale;
  d.residual_scale = p.residual_scale;
  const int64_t grid = (p.N + kRows - 1) / kRows;
  // Four steps of K a warp at least, where there are that many.
  d.warps = 1;
  while (d.warps < kWarps && d.warps * 128 < p.K) d.warps *= 2;
  // Where K is so long that outputs have the bits to show it: sums of 768 in fp32, of 262,144 in bf16.  In
  // segments 1 x 4096 x 6144 would take 12.2 us, not 12.0, and 16 x 2048 x 4096 6.6, not 6.2.
  const bool f32 = p.out.type == ENGRAM_DTYPE_F32 || (p.pre.p && p.pre.type == ENGRAM_DTYPE_F32);
  const bool segments = p.K > (int64_t)d.warps * 2 * (f32 ? kSegment * 16 : 262144);
  if (p.M <= 8) return segments ? launch_eights<1, true>(d, grid, stream) : launch_eights<1, false>(d, grid, stream);
  return segments ? launch_eights<2, true>(d, grid, stream) : launch_eights<2, false>(d, grid, stream);
}

}  // namespace engram

// fp8_quantise.cu -- e4m3 values with one power-of-two scale per block of 128.
//
// A block B (128 values along a row, or a 128 x 128 tile) gets the smallest exponent
// e >= -127 with max|B| <= 448 * 2^e, stored as the byte e + 127 (OCP E8M0), and its
// values become e4m3(x 2^-e), rounded to nearest even.  The scale being a power of two,
// x 2^-e is exact in fp32: the only rounding is the one to e4m3, and the matrix product
// can hand the byte to the tensor cores as it is.  With max|B| = m 2^x, 1 <= m < 2, and
// 448 = 1.75 * 2^8, e = x - 8, or x - 7 when m > 1.75: integer arithmetic on the bits of
// the maximum.  Magnitudes are compared as integers, so a NaN or infinity wins; such a
// block gets the NaN scale 0xFF and NaN bytes 0x7F.
//
// HBM-bound: x read once, a byte a value written (two with the transposed copy).
//   rows kernel: 16 lanes a block of 128 values (8 each), four blocks of loads in
//     flight a thread;
//   tile kernel (a transposed copy, or 128 x 128 blocks): a 128 x 128 tile in the
//     registers of 256 threads -- 16 rows x 4 columns each, so row maxima are warp
//     reductions and column maxima one exchange through shared memory; the transposed
//     bytes are turned in shared memory (16 KB, chunks of 16 bytes XOR-swizzled by the
//     column) so that both copies leave as whole 128-byte lines.  Two persistent blocks an
//     SM walk the tiles; a tile comes by one tensor copy into shared memory, and as soon as
//     it is in registers the next one's copy starts, under its arithmetic.
#include <cuda_fp8.h>

#include <atomic>

#include "launch.cuh"
#include "lookup_common.cuh"
#include "tensor_core.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr uint32_t kNaN4 = 0x7F7F7F7Fu;

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int32_t x = (int32_t)(bits >> 23);
  if (x == 255) return 255;  // NaN or infinity
  const int32_t e = x - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  return e < 0 ? 0 : (uint32_t)e;
}

// 2^(127 - s): what a block's values are multiplied by (s in [0, 247]: a normal number).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, uint32_t s) {
  if (s == 255) return kNaN4;
  const float m = inverse_scale(s);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * m, b * m), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * m, d * m), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ uint32_t mag(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// N values of a row from column `col` on, zero beyond K.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_vals(const T *row, int64_t col, int64_t K, float (&f)[N]) {
  if constexpr (VEC) {
    if (col + N <= K) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
          const float4 v = __ldcs(reinterpret_cast<const float4 *>(row + col) + i);
          f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
          const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(row + col) + i);
          f[4 * i] = bf16_lo(v.x), f[4 * i + 1] = bf16_hi(v.x);
          f[4 * i + 2] = bf16_lo(v.y), f[4 * i + 3] = bf16_hi(v.y);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = 0.f;
    if (col + i < K) {
      if constexpr (sizeof(T) == 4)
        f[i] = __ldg(row + col + i);
      else
        f[i] = bf16_lo(__ldg(row + col + i));
    }
  }
}

constexpr int kRowsThreads = 256;

template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(kRowsThreads)
    quantise_rows_kernel(const __grid_constant__ QuantiseParams p, int32_t kblocks) {
  dependency_wait();
  const int64_t n = p.M * kblocks;
  const int in = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * (kRowsThreads / 16 * U) + (threadIdx.x >> 4);
  float f[U][8];
  int64_t row[U], col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b = first + u * (kRowsThreads / 16);
    row[u] = b < n ? b / kblocks : -1;
    col[u] = b < n ? (b - row[u] * kblocks) * 128 + in * 8 : 0;
    if (row[u] >= 0)
      load_vals<T, 8, VEC>(static_cast<const T *>(p.x) + row[u] * p.x_stride, col[u], p.K, f[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = 0;
    if (row[u] >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mag(f[u][i]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (row[u] < 0) continue;
    const uint32_t s = scale_byte(m);
    if (in == 0) p.s[row[u] * kblocks + (col[u] >> 7)] = (uint8_t)s;
    const uint2 w = make_uint2(quantise4(f[u][0], f[u][1], f[u][2], f[u][3], s),
                               quantise4(f[u][4], f[u][5], f[u][6], f[u][7], s));
    uint8_t *q = p.q + row[u] * p.q_stride + col[u];
    if (col[u] + 8 <= p.K) {
      *reinterpret_cast<uint2 *>(q) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col[u] + i < p.K) q[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

// The tile (mb, kb), held as 16 rows x 4 columns a thread: its scales and bytes.
__device__ __forceinline__ void quantise_tile(const QuantiseParams &p, const float (&v)[16][4], int64_t mb,
                                              int64_t kb, int32_t kblocks, int32_t mblocks, uint4 *s_turn,
                                              uint4 (*s_max)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m0 = mb * 128 + warp * 16, k0 = kb * 128 + lane * 4;
  // Column maxima: this thread's 16 rows, then the eight warps' through shared memory.
  uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[j] = max(cm[j], mag(v[i][j]));
  s_max[warp][lane] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const uint4 o = s_max[w][lane];
    cm[0] = max(cm[0], o.x), cm[1] = max(cm[1], o.y);
    cm[2] = max(cm[2], o.z), cm[3] = max(cm[3], o.w);
  }
  uint32_t tile = 0;
  if (p.block_rows != 1) {
    tile = max(max(cm[0], cm[1]), max(cm[2], cm[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tile = max(tile, __shfl_xor_sync(0xffffffffu, tile, o));
    tile = scale_byte(tile);
    if (threadIdx.x == 0) {
      if (p.s) p.s[mb * kblocks + kb] = (uint8_t)tile;
      if (p.st) p.st[kb * mblocks + mb] = (uint8_t)tile;
    }
  }
  if (p.q) {
    uint32_t rs = tile;  // lanes 2i and 2i + 1: row i's scale
    if (p.block_rows == 1) {
      // Row maxima: 16 values a lane, halved in number at each of four exchanges.
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        r[i] = max(max(mag(v[i][0]), mag(v[i][1])), max(mag(v[i][2]), mag(v[i][3])));
#pragma unroll
      for (int half = 8; half > 0; half >>= 1) {
        const bool up = lane & (2 * half);
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const uint32_t give = up ? r[i] : r[i + half], keep = up ? r[i + half] : r[i];
          r[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, 2 * half));
        }
      }
      r[0] = max(r[0], __shfl_xor_sync(0xffffffffu, r[0], 1));
      rs = scale_byte(r[0]);
      const int64_t row = m0 + (lane >> 1);
      if (!(lane & 1) && row < p.M) p.s[row * kblocks + kb] = (uint8_t)rs;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t s = __shfl_sync(0xffffffffu, rs, 2 * i);
      if (m0 + i < p.M) {
        const uint32_t w = quantise4(v[i][0], v[i][1], v[i][2], v[i][3], s);
        uint8_t *q = p.q + (m0 + i) * p.q_stride + k0;
        if (k0 + 4 <= p.K) {
          *reinterpret_cast<uint32_t *>(q) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k0 + j < p.K) q[j] = (uint8_t)(w >> (8 * j));
        }
      }
    }
  }
  if (p.qt) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s = p.block_rows == 1 ? scale_byte(cm[j]) : tile;
      if (p.block_rows == 1 && warp == 0 && k0 + j < p.K) p.st[(k0 + j) * mblocks + mb] = (uint8_t)s;
      uint4 w;
      w.x = quantise4(v[0][j], v[1][j], v[2][j], v[3][j], s);
      w.y = quantise4(v[4][j], v[5][j], v[6][j], v[7][j], s);
      w.z = quantise4(v[8][j], v[9][j], v[10][j], v[11][j], s);
      w.w = quantise4(v[12][j], v[13][j], v[14][j], v[15][j], s);
      s_turn[(lane * 4 + j) * 8 + (warp ^ (lane & 7))] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = i * 256 + threadIdx.x;
      const int c = idx >> 3, chunk = idx & 7;
      const int64_t k = kb * 128 + c, m = mb * 128 + chunk * 16;
      if (k >= p.K || m >= p.M) continue;
      const uint4 w = s_turn[c * 8 + (chunk ^ ((c >> 2) & 7))];
      uint8_t *q = p.qt + k * p.qt_stride + m;
      if (m + 16 <= p.M) {
        *reinterpret_cast<uint4 *>(q) = w;
      } else {
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (m + e < p.M) q[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
}

// A tile loaded into registers, for rows that are not on 16-byte boundaries.
template <typename T>
__global__ void __launch_bounds__(256, 2)
    quantise_tile_kernel(const __grid_constant__ QuantiseParams p, int32_t kblocks, int32_t mblocks) {
  __shared__ uint4 s_turn[128 * 8];
  __shared__ uint4 s_max[8][32];  // [warp][lane]: the maxima of four columns
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t mb = blockIdx.x / kblocks, kb = blockIdx.x - mb * kblocks;
  const int64_t m0 = mb * 128 + warp * 16, k0 = kb * 128 + lane * 4;
  float v[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (m0 + i < p.M) {
      load_vals<T, 4, false>(static_cast<const T *>(p.x) + (m0 + i) * p.x_stride, k0, p.K, v[i]);
    } else {
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
    }
  }
  quantise_tile(p, v, mb, kb, kblocks, mblocks, s_turn, s_max);
}

template <typename T>
__global__ void __launch_bounds__(256, 2)
    quantise_tma_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ QuantiseParams p,
                        int32_t kblocks, int32_t mblocks) {
  extern __shared__ __align__(128) uint8_t s_tile[];  // [128 rows][128 values], zero outside x
  __shared__ uint4 s_turn[128 * 8];
  __shared__ uint4 s_max[8][32];
  __shared__ uint64_t s_full;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t tiles = kblocks * mblocks;  // under 2^31
  constexpr uint32_t kRow = 128 * sizeof(T);
  if (tid == 0) {
    mbar_init(&s_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  dependency_wait();
  __syncthreads();
  int32_t mb = (int32_t)blockIdx.x / kblocks, kb = (int32_t)blockIdx.x - mb * kblocks;
  const auto issue = [&](int32_t m, int32_t k) {
    mbar_arrive_expect_tx(&s_full, 128 * kRow);
    tma_load_2d(s_tile, &map, k * 128, m * 128, &s_full);
  };
  if (tid == 0 && (int32_t)blockIdx.x < tiles) issue(mb, kb);
  uint32_t phase = 0;
  for (int32_t tile = blockIdx.x; tile < tiles; phase ^= 1) {
    const bool late = !drain_phase(&s_full, phase, p.wait_limit_ns);
    float v[16][4];
    const T *src = reinterpret_cast<const T *>(s_tile + warp * 16 * kRow) + lane * 4;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(src + i * 128);
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(src + i * 128);
        v[i][0] = bf16_lo(w.x), v[i][1] = bf16_hi(w.x), v[i][2] = bf16_lo(w.y), v[i][3] = bf16_hi(w.y);
      }
    }
    if (__syncthreads_or(late)) {  // the copy did not arrive: the block stops together
      if (tid == 0) {
        if (p.status) atomicOr(p.status, ENGRAM_FLAG_TIMEOUT);
        drain_phase(&s_full, phase, p.wait_limit_ns);  // it lands, or gives up likewise
      }
      break;
    }
    const int32_t this_mb = mb, this_kb = kb;
    tile += gridDim.x;
    mb = tile / kblocks, kb = tile - mb * kblocks;
    if (tid == 0 && tile < tiles) issue(mb, kb);
    quantise_tile(p, v, this_mb, this_kb, kblocks, mblocks, s_turn, s_max);
  }
}

// x as a 2-D tiled map with box [128 values, 128 rows], zero fill outside.
template <typename T>
bool make_map(CUtensorMap *map, const QuantiseParams &p) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)p.M};
  const cuuint64_t strides[1] = {(cuuint64_t)(p.x_stride * sizeof(T))};
  const cuuint32_t box[2] = {128, 128}, estr[2] = {1, 1};
  return fn(map, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void *>(p.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t launch_typed(const QuantiseParams &p, cudaStream_t stream) {
  const int64_t kblocks = (p.K + 127) / 128, mblocks = (p.M + 127) / 128;
  if (!p.qt && p.block_rows == 1) {
    const bool vec = (uintptr_t)p.x % 16 == 0 && p.x_stride * sizeof(T) % 16 == 0;
    const int64_t n = p.M * kblocks;
    constexpr int kPer = kRowsThreads / 16;
    if (n <= 152 * 8 * kPer) {
      const int64_t grid = (n + kPer - 1) / kPer;
      if (vec)
        return launch(quantise_rows_kernel<T, true, 1>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks);
      else
        return launch(quantise_rows_kernel<T, false, 1>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks);
    } else {
      const int64_t grid = (n + kPer * 4 - 1) / (kPer * 4);
      if (vec)
        return launch(quantise_rows_kernel<T, true, 4>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks);
      else
        return launch(quantise_rows_kernel<T, false, 4>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks);
    }
  } else {
    const int64_t tiles = kblocks * mblocks;
    const int64_t stride = p.M > 1 ? p.x_stride : (p.K + 7) / 8 * 8;  // one row needs none
    if ((uintptr_t)p.x % 16 != 0 || stride * sizeof(T) % 16 != 0)
      return launch(quantise_tile_kernel<T>, tiles, 256, 0, stream, 1, p, (int32_t)kblocks, (int32_t)mblocks);
    constexpr int kTileBytes = 128 * 128 * sizeof(T);
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(configured.load(std::memory_order_relaxed) & 1ull << (dev & 63))) {
      e = cudaFuncSetAttribute(quantise_tma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
      if (e != cudaSuccess) return e;
      configured.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    QuantiseParams q = p;
    q.x_stride = stride;
    CUtensorMap map;
    if (!make_map<T>(&map, q)) return cudaErrorInvalidValue;
    const int64_t grid = tiles < 2 * kSms ? tiles : 2 * kSms;
    return launch(quantise_tma_kernel<T>, grid, 256, kTileBytes, stream, 1, map, p, (int32_t)kblocks,
                  (int32_t)mblocks);
  }
}

}  // namespace

cudaError_t launch_quantise(const QuantiseParams &p, int dtype, cudaStream_t stream) {
  return dtype == ENGRAM_DTYPE_F32 ? launch_typed<float>(p, stream) : launch_typed<uint16_t>(p, stream);
}

}  // namespace engram

// fp8_quantise.cu -- e4m3 values with one power-of-two scale per block of 128.
//
// A block B (128 values along a row, or a 128 x 128 tile) gets the smallest exponent
// e >= -127 with max|B| <= 448 * 2^e, stored as the byte e + 127 (OCP E8M0), and its
// values become e4m3(x 2^-e), rounded to nearest even.  The scale being a power of two,
// x 2^-e is exact in fp32: the only rounding is the one to e4m3, and the matrix product
// can hand the byte to the tensor cores as it is.  With max|B| = m 2^x, 1 <= m < 2, and
// 448 = 1.75 * 2^8, e = x - 8, or x - 7 when m > 1.75: integer arithmetic on the bits of
// the maximum.  The maximum keeps NaN, and a NaN or infinity gives its block the NaN
// scale 0xFF and NaN bytes 0x7F.
//
// HBM-bound: x read once, a byte a value written (two with the transposed copy).
//   linear kernel (x and q without gaps, K a multiple of 128: block b is values 128 b ..):
//     8 lanes a block, 16 values each in two runs of 8, one block a thread;
//   rows kernel (any strides and widths): 16 lanes a block, 8 values each; rows off 16-byte
//     boundaries come value by value (65,536 x 4096 fp32 with gaps: 194 us, its bytes at the
//     copy bandwidth; x 4099: 275 us of 201, bf16 264 of 121);
//   tile kernel (a transposed copy, or 128 x 128 blocks): a 128 x 128 tile in the
//     registers of 256 threads -- 16 rows x 4 columns each, so row maxima are warp
//     reductions and column maxima one exchange through shared memory; the transposed
//     bytes are turned in shared memory (16 KB, chunks of 16 bytes XOR-swizzled by the
//     column) so that both copies leave as whole 128-byte lines.  Two persistent blocks an
//     SM walk the tiles; a tile comes by one tensor copy into shared memory, and as soon as
//     it is in registers the next one's copy starts, under its arithmetic.  Rows off 16-byte
//     boundaries: a tile a block, loaded value by value (65,536 x 4099, both copies: fp32 333
//     us of 241, bf16 705 of 161).
#include <cuda_fp8.h>

#include <atomic>

#include "launch.cuh"
#include "lookup_common.cuh"
#include "tensor_core.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int32_t x = (int32_t)(bits >> 23);
  if (x == 255) return 255;  // NaN or infinity
  const int32_t e = x - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  return e < 0 ? 0 : (uint32_t)e;
}

// 2^(127 - s): what a block's values are multiplied by (s in [0, 247]: a normal number).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// What a block's values are multiplied by: NaN for the NaN scale, so that they become NaN.
__device__ __forceinline__ float multiplier(uint32_t s) {
  return s == 255 ? __uint_as_float(0x7FFFFFFFu) : inverse_scale(s);
}

__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, float m) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * m, b * m), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * m, d * m), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The larger magnitude; NaN if either is NaN (its exponent then marks the block).
__device__ __forceinline__ float max_mag(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}
__device__ __forceinline__ uint32_t scale_byte(float largest) {
  return scale_byte(__float_as_uint(largest) & 0x7FFFFFFFu);
}

template <int N>
__device__ __forceinline__ float max_of(const float (&f)[N]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = max_mag(m, f[i]);
  return m;
}

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
        static_assert(sizeof(T) == 4 || N == 8);
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + col));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
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

template <typename T>
__global__ void __launch_bounds__(kRowsThreads) quantise_linear_kernel(const __grid_constant__ QuantiseParams p,
                                                                       int64_t n) {
  dependency_wait();
  const int in = threadIdx.x & 7;
  const int64_t b = (int64_t)blockIdx.x * (kRowsThreads / 8) + (threadIdx.x >> 3), at = b * 128 + in * 8;
  float lo[8], hi[8];  // zero past the last block
  load_vals<T, 8, true>(static_cast<const T *>(p.x), at, n * 128, lo);
  load_vals<T, 8, true>(static_cast<const T *>(p.x), at + 64, n * 128, hi);
  float m = max_mag(max_of<8>(lo), max_of<8>(hi));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (b >= n) return;
  const uint32_t s = scale_byte(m);
  if (in == 0) p.s[b] = (uint8_t)s;
  const float by = multiplier(s);
  uint2 *q = reinterpret_cast<uint2 *>(p.q + at);
  q[0] = make_uint2(quantise4(lo[0], lo[1], lo[2], lo[3], by), quantise4(lo[4], lo[5], lo[6], lo[7], by));
  q[8] = make_uint2(quantise4(hi[0], hi[1], hi[2], hi[3], by), quantise4(hi[4], hi[5], hi[6], hi[7], by));
}

// Blocks of 128 values numbered along the rows, 16 lanes each, U of them a thread.  A thread
// block's local numbers x are below kblocks + 16 U.  Short rows take x / kblocks by `magic` =
// ceil(2^32 / kblocks), exact while x (magic kblocks - 2^32) < x kblocks < 2^32, so far beyond
// kblocks = 16 U; from there on a thread block meets one row's end at most, and a comparison
// does for rows of any length.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(kRowsThreads)
    quantise_rows_kernel(const __grid_constant__ QuantiseParams p, int32_t kblocks, uint32_t magic) {
  dependency_wait();
  constexpr int kPer = kRowsThreads / 16;
  const int in = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t base = (int64_t)blockIdx.x * (kPer * U);
  const int64_t row0 = base / kblocks;
  const uint32_t rem0 = (uint32_t)(base - row0 * kblocks);
  float f[U][8];
  int64_t row[U];
  int32_t kb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t x = rem0 + u * kPer + slot;
    const uint32_t q = kblocks >= kPer * U ? x >= (uint32_t)kblocks : kblocks == 1 ? x : __umulhi(x, magic);
    row[u] = row0 + q;
    kb[u] = (int32_t)(x - q * kblocks);
    if (row[u] < p.M)
      load_vals<T, 8, VEC>(static_cast<const T *>(p.x) + row[u] * p.x_stride, (int64_t)kb[u] * 128 + in * 8, p.K,
                           f[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = 0.f;
    if (row[u] < p.M) {
      m = max_of<8>(f[u]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (row[u] >= p.M) continue;
    const uint32_t s = scale_byte(m);
    if (in == 0) p.s[row[u] * kblocks + kb[u]] = (uint8_t)s;
    const float by = multiplier(s);
    const uint2 w = make_uint2(quantise4(f[u][0], f[u][1], f[u][2], f[u][3], by),
                               quantise4(f[u][4], f[u][5], f[u][6], f[u][7], by));
    const int64_t col = (int64_t)kb[u] * 128 + in * 8;
    uint8_t *q = p.q + row[u] * p.q_stride + col;
    if (col + 8 <= p.K) {
      *reinterpret_cast<uint2 *>(q) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < p.K) q[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

// The tile kernel's arithmetic in two forms that give the same bytes.  LEAN: maxima by
// max.NaN on the values, the NaN scale as a multiplier, edges looked up once a tile.  The
// other one, with integer maxima and a branch per word, issues about a third more
// instructions.  bf16 tiles, which the arithmetic binds, take LEAN (24,935 x 1664 with 128 x
// 128 blocks, both copies: 31 us against 44); fp32 tiles, which HBM binds, the other
// (65,536 x 4096, both copies: 265 us against 284; why the longer form's pace suits HBM
// better is not established).
template <bool LEAN>
struct Form {
  static __device__ __forceinline__ uint32_t larger(uint32_t bits, float f) {
    if constexpr (LEAN) return __float_as_uint(max_mag(__uint_as_float(bits), f));
    return max(bits, __float_as_uint(f) & 0x7FFFFFFFu);
  }
  // What quantise() takes for a block of scale byte s.
  static __device__ __forceinline__ uint32_t code(uint32_t s) {
    if constexpr (LEAN) return __float_as_uint(multiplier(s));
    return s;
  }
  static __device__ __forceinline__ uint32_t quantise(float a, float b, float c, float d, uint32_t code) {
    if constexpr (LEAN) return quantise4(a, b, c, d, __uint_as_float(code));
    if (code == 255) return 0x7F7F7F7Fu;
    return quantise4(a, b, c, d, inverse_scale(code));
  }
};

// The tile (mb, kb), held as 16 rows x 4 columns a thread: its scales and bytes.
template <bool LEAN>
__device__ __forceinline__ void quantise_tile(const QuantiseParams &p, const float (&v)[16][4], int64_t mb,
                                              int64_t kb, int32_t kblocks, int32_t mblocks, uint4 *s_turn,
                                              uint4 (*s_max)[32]) {
  using F = Form<LEAN>;
  const auto join = [](uint32_t x, uint32_t y) { return F::larger(x, __uint_as_float(y)); };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m0 = mb * 128 + warp * 16, k0 = kb * 128 + lane * 4;
  const bool whole = LEAN && (mb + 1) * 128 <= p.M && (kb + 1) * 128 <= p.K;  // no edge to look out for
  // Column maxima: this thread's 16 rows, then the eight warps' through shared memory.
  uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[j] = F::larger(cm[j], v[i][j]);
  s_max[warp][lane] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const uint4 o = s_max[w][lane];
    cm[0] = join(cm[0], o.x), cm[1] = join(cm[1], o.y);
    cm[2] = join(cm[2], o.z), cm[3] = join(cm[3], o.w);
  }
  uint32_t tile = 0;
  if (p.block_rows != 1) {
    tile = join(join(cm[0], cm[1]), join(cm[2], cm[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tile = join(tile, __shfl_xor_sync(0xffffffffu, tile, o));
    tile = scale_byte(tile);
    if (threadIdx.x == 0) {
      if (p.s) p.s[mb * kblocks + kb] = (uint8_t)tile;
      if (p.st) p.st[kb * mblocks + mb] = (uint8_t)tile;
    }
  }
  if (p.q) {
    uint32_t by = F::code(tile);  // lanes 2i and 2i + 1: row i's
    if (p.block_rows == 1) {
      // Row maxima: 16 values a lane, halved in number at each of four exchanges.
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        r[i] = F::larger(F::larger(0, v[i][0]), v[i][1]);
        r[i] = join(r[i], F::larger(F::larger(0, v[i][2]), v[i][3]));
      }
#pragma unroll
      for (int half = 8; half > 0; half >>= 1) {
        const bool up = lane & (2 * half);
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const uint32_t give = up ? r[i] : r[i + half], keep = up ? r[i + half] : r[i];
          r[i] = join(keep, __shfl_xor_sync(0xffffffffu, give, 2 * half));
        }
      }
      r[0] = join(r[0], __shfl_xor_sync(0xffffffffu, r[0], 1));
      const uint32_t rs = scale_byte(r[0]);
      by = F::code(rs);
      const int64_t row = m0 + (lane >> 1);
      if (!(lane & 1) && row < p.M) p.s[row * kblocks + kb] = (uint8_t)rs;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t row_by = __shfl_sync(0xffffffffu, by, 2 * i);
      if (whole || m0 + i < p.M) {
        const uint32_t w = F::quantise(v[i][0], v[i][1], v[i][2], v[i][3], row_by);
        uint8_t *q = p.q + (m0 + i) * p.q_stride + k0;
        if (whole || k0 + 4 <= p.K) {
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
      const uint32_t by = F::code(s);
      uint4 w;
      w.x = F::quantise(v[0][j], v[1][j], v[2][j], v[3][j], by);
      w.y = F::quantise(v[4][j], v[5][j], v[6][j], v[7][j], by);
      w.z = F::quantise(v[8][j], v[9][j], v[10][j], v[11][j], by);
      w.w = F::quantise(v[12][j], v[13][j], v[14][j], v[15][j], by);
      s_turn[(lane * 4 + j) * 8 + (warp ^ (lane & 7))] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = i * 256 + threadIdx.x;
      const int c = idx >> 3, chunk = idx & 7;
      const int64_t k = kb * 128 + c, m = mb * 128 + chunk * 16;
      if (!whole && (k >= p.K || m >= p.M)) continue;
      const uint4 w = s_turn[c * 8 + (chunk ^ ((c >> 2) & 7))];
      uint8_t *q = p.qt + k * p.qt_stride + m;
      if (whole || m + 16 <= p.M) {
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
  quantise_tile<true>(p, v, mb, kb, kblocks, mblocks, s_turn, s_max);
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
  if (tid == 0 && (int32_t)blockIdx.x < tiles) {
    if (p.withhold)
      mbar_arrive_expect_tx(&s_full, 128 * kRow);
    else
      issue(mb, kb);
  }
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
    quantise_tile<sizeof(T) == 2>(p, v, this_mb, this_kb, kblocks, mblocks, s_turn, s_max);
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
    if (vec && p.K % 128 == 0 && (p.M == 1 || (p.x_stride == p.K && p.q_stride == p.K))) {
      return launch(quantise_linear_kernel<T>, (n * 8 + kRowsThreads - 1) / kRowsThreads, kRowsThreads, 0, stream, 1,
                    p, n);
    }
    const uint32_t magic = (uint32_t)(((1ull << 32) + kblocks - 1) / kblocks);
    if (n <= kSms * 8 * kPer) {
      const int64_t grid = (n + kPer - 1) / kPer;
      if (vec)
        return launch(quantise_rows_kernel<T, true, 1>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks, magic);
      else
        return launch(quantise_rows_kernel<T, false, 1>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks, magic);
    } else {
      const int64_t grid = (n + kPer * 4 - 1) / (kPer * 4);
      if (vec)
        return launch(quantise_rows_kernel<T, true, 4>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks, magic);
      else
        return launch(quantise_rows_kernel<T, false, 4>, grid, kRowsThreads, 0, stream, 1, p, (int32_t)kblocks, magic);
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
    q.withhold = take_withheld_launch();
    const int64_t grid = tiles < 2 * kSms ? tiles : 2 * kSms;
    return launch(quantise_tma_kernel<T>, grid, 256, kTileBytes, stream, 1, map, q, (int32_t)kblocks,
                  (int32_t)mblocks);
  }
}

}  // namespace

cudaError_t launch_quantise(const QuantiseParams &p, int dtype, cudaStream_t stream) {
  return dtype == ENGRAM_DTYPE_F32 ? launch_typed<float>(p, stream) : launch_typed<uint16_t>(p, stream);
}

}  // namespace engram

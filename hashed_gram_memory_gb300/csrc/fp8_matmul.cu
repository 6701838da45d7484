// fp8_matmul.cu -- out[m, n] = sum_k a[m, k] b[n, k], both e4m3 with one power-of-two
// scale per block of 128 along K, on the sm_103a tensor cores.
//
// tcgen05.mma kind::mxf8f6f4 multiplies each 32-wide slice of products by one E8M0 scale
// per row of A and of B before it adds them to the fp32 accumulator, so a block of 128 is
// four instructions reading the same scale byte: no pass over the accumulator per block.
// The roles are turned around: the rows of b (the output's columns) are the instruction's
// M rows, the rows of a its N columns, so that a warp of the epilogue holds 32
// neighbouring outputs of one row of out in its lanes and stores whole lines for any
// output stride and size.
//
// One persistent CTA per SM walks 128 (b) x up to 128 (a) tiles.  Warps:
//   0     TMA producer: a ring of stages, each a 128-byte slice along K of the tile's rows
//         of a and b (128-byte swizzle);
//   1     allocates TMEM; one thread copies the scales to TMEM (tcgen05.cp) and issues the
//         MMAs into one of two accumulators;
//   2..5  epilogue: TMEM lanes 32*(warp%4).., stores;
//   6     scales: for every four blocks of K one 32-bit word per row, put into shared
//         memory in the order tcgen05.cp wants (word (r%32)*4 + r/32 of each 128 rows).
// Every wait is bounded as in wkv_gemm.cu: one that gives up sets ENGRAM_FLAG_TIMEOUT and
// leaves the tiles not yet stored unwritten.
#include <mutex>

#include "lookup_common.cuh"
#include "tensor_core.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr int kP = 128;       // rows of b a tile
constexpr int kQMax = 128;    // most rows of a a tile
constexpr int kThreads = 224;
constexpr int kScaleSlots = 4;
constexpr uint32_t kSlotBytes = (kP + kQMax) * 4;
constexpr int kMaxStages = 8;
constexpr uint32_t kStageBudget = 192 * 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 2 * kQMax;  // scale words: two buffers of 4 (b) + 4 (a) columns
constexpr size_t kSmemBytes = 1024 + kStageBudget + kScaleSlots * kSlotBytes + 512;

struct MatmulDev {
  const uint8_t *a_scale, *b_scale;
  void *out;
  int32_t *status;
  int64_t M, N, out_stride;
  int32_t kblocks, a_shift, b_shift;  // log2 of the rows sharing a scale (0 or 7)
  int32_t q_tile, stages;
  int64_t tiles_q, tiles;
  int64_t wait_limit_ns;
};

// Shared-memory descriptor of the scale words: 32 rows of 16 bytes, no swizzle, 8-row
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 |
         (uint64_t)1 << 46;
}

// Instruction descriptor of kind::mxf8f6f4: e4m3 operands, both K-major, UE8M0 scales;
// bits 4-5 and 29-30 choose the byte of the scale words.
__device__ __forceinline__ uint32_t instr_desc(uint32_t m, uint32_t n, uint32_t byte) {
  return byte << 4 | (n >> 3) << 17 | 1u << 23 | (m >> 7) << 27 | byte << 29;
}

__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t p_desc, uint64_t q_desc, uint32_t idesc,
                                         uint32_t sp, uint32_t sq, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(p_desc), "l"(q_desc), "r"(idesc), "r"(sp), "r"(sq), "r"(accumulate)
      : "memory");
}

// The scale bytes of four blocks of K (from block kb on) of one row, zero past either end.
__device__ __forceinline__ uint32_t scale_word(const uint8_t *s, int64_t row, int64_t rows, int shift,
                                               int kb, int kblocks) {
  if (row >= rows) return 0;
  const uint8_t *src = s + (row >> shift) * kblocks + kb;
  if (kb + 4 <= kblocks && ((uintptr_t)src & 3) == 0) return __ldg(reinterpret_cast<const uint32_t *>(src));
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (kb + i < kblocks) w |= (uint32_t)__ldg(src + i) << (8 * i);
  return w;
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

template <typename TO>
__device__ __forceinline__ void store_out(TO *dst, uint32_t v) {
  if constexpr (sizeof(TO) == 4)
    *dst = __uint_as_float(v);
  else
    *dst = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v)));
}

template <typename TO>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ MatmulDev p) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t *slots = sm + kStageBudget;
  uint64_t *full = reinterpret_cast<uint64_t *>(slots + kScaleSlots * kSlotBytes);
  uint64_t *empty = full + kMaxStages;
  uint64_t *sc_full = empty + kMaxStages;
  uint64_t *sc_empty = sc_full + kScaleSlots;
  uint64_t *acc_full = sc_empty + kScaleSlots;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks = p.kblocks, stages = p.stages, qt = p.q_tile;
  const uint32_t stage_bytes = (uint32_t)(kP + qt) * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(sc_full + s, 1);
      mbar_init(sc_empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full + a, 1);
      mbar_init(acc_empty + a, 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- TMA producer
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
        const int p0 = (int)(tile / p.tiles_q) * kP, q0 = (int)(tile % p.tiles_q) * qt;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          if (!(ok = wait_phase(empty + s, ph ^ 1, abort_flag, p.wait_limit_ns, p.status))) break;
          uint8_t *st = sm + s * stage_bytes;
          mbar_arrive_expect_tx(full + s, stage_bytes);
          tma_load_2d(st, &map_b, kb * 128, p0, full + s);
          tma_load_2d(st + kP * 128, &map_a, kb * 128, q0, full + s);
          if (++s == stages) s = 0, ph ^= 1;
        }
      }
      // Loads issued into shared memory land before the block can exit.
      for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j)
        drain_phase(full + j % stages, (j / stages) & 1, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      uint32_t local = 0, group = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x, ++local) {
        const uint32_t acc = local & 1, use = local >> 1;
        if (!wait_phase(acc_empty + acc, (use & 1) ^ 1, abort_flag, p.wait_limit_ns, p.status)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + acc * kQMax;
        uint32_t sp = 0, sq = 0;
        for (int kb = 0; kb < kblocks; ++kb) {
          if ((kb & 3) == 0) {  // the scales of the next four blocks
            const int slot = group % kScaleSlots;
            if (!(ok = wait_phase(sc_full + slot, (group / kScaleSlots) & 1, abort_flag,
                                  p.wait_limit_ns, p.status)))
              break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            sp = tmem + kScaleCol + (group & 1) * 8, sq = sp + 4;
            const uint32_t src = smem_u32(slots + slot * kSlotBytes);
            copy_scales(sp, smem_desc_scales(src));
            copy_scales(sq, smem_desc_scales(src + kP * 4));
            umma_commit(sc_empty + slot);
            ++group;
          }
          if (!(ok = wait_phase(full + s, ph, abort_flag, p.wait_limit_ns, p.status))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t ps = smem_u32(sm + s * stage_bytes), qs = ps + kP * 128;
          const uint32_t idesc = instr_desc(kP, qt, kb & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_fp8(d, smem_desc_sw128(ps + 32 * k), smem_desc_sw128(qs + 32 * k), idesc, sp, sq,
                     (kb | k) != 0 ? 1u : 0u);
          umma_commit(empty + s);
          if (++s == stages) s = 0, ph ^= 1;
        }
        if (ok) umma_commit(acc_full + acc);
      }
      umma_commit(mma_done);
    }
  } else if (warp == 6) {
    // --------------------------------------------------------------- scales
    uint32_t group = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
      const int64_t p0 = tile / p.tiles_q * kP, q0 = tile % p.tiles_q * qt;
      for (int kb = 0; kb < kblocks; kb += 4, ++group) {
        const int slot = group % kScaleSlots;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = scale_word(p.b_scale, p0 + 32 * i + lane, p.N, p.b_shift, kb, kblocks);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[4 + i] = 32 * i < qt ? scale_word(p.a_scale, q0 + 32 * i + lane, p.M, p.a_shift, kb, kblocks) : 0;
        ok = __all_sync(0xffffffffu, wait_phase(sc_empty + slot, ((group / kScaleSlots) & 1) ^ 1,
                                                abort_flag, p.wait_limit_ns, p.status));
        if (!ok) break;
        uint4 *dst = reinterpret_cast<uint4 *>(slots + slot * kSlotBytes);
        dst[lane] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[32 + lane] = make_uint4(w[4], w[5], w[6], w[7]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full + slot);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    uint32_t local = 0;
    for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, ++local) {
      const uint32_t acc = local & 1, use = local >> 1;
      const bool ok = wait_phase(acc_full + acc, use & 1, abort_flag, p.wait_limit_ns, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int64_t n = tile / p.tiles_q * kP + quad * 32 + lane;
      const int64_t m0 = tile % p.tiles_q * qt;
      TO *out = static_cast<TO *>(p.out) + n;
#pragma unroll 1
      for (int c = 0; c < qt; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + acc * kQMax + c, v);
        if (n < p.N) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (m0 + c + i < p.M) store_out(out + (m0 + c + i) * p.out_stride, v[i]);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + acc);
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) drain_phase(mma_done, 0, p.wait_limit_ns);
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

// A row-major byte matrix [rows, cols] with rows `stride` apart as a 2-D tiled map with
// box [128 bytes, box_rows], 128-byte swizzle, zero fill outside.
bool make_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t stride,
              uint32_t box_rows) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceInfo {
  bool ready = false;
  int sms = 0;
};
DeviceInfo g_info[64];
std::mutex g_info_mu;

cudaError_t device_info(DeviceInfo &out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_info_mu);
  DeviceInfo &d = g_info[dev & 63];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (auto *k : {fp8_matmul_kernel<float>, fp8_matmul_kernel<uint16_t>})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    d.ready = true;
  }
  out = d;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_fp8_matmul(const MatmulParams &p, int out_dtype, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(info);
  if (e != cudaSuccess) return e;
  MatmulDev d{};
  d.a_scale = p.a_scale;
  d.b_scale = p.b_scale;
  d.out = p.out;
  d.status = p.status;
  d.M = p.M;
  d.N = p.N;
  d.out_stride = p.out_stride;
  d.kblocks = (int32_t)((p.K + 127) / 128);
  d.a_shift = p.a_block == 1 ? 0 : 7;
  d.b_shift = p.b_block == 1 ? 0 : 7;
  d.q_tile = (int32_t)(p.M < kQMax ? (p.M + 15) / 16 * 16 : kQMax);
  d.stages = (int32_t)(kStageBudget / ((kP + d.q_tile) * 128));
  if (d.stages > kMaxStages) d.stages = kMaxStages;
  d.tiles_q = (p.M + d.q_tile - 1) / d.q_tile;
  d.tiles = d.tiles_q * ((p.N + kP - 1) / kP);
  d.wait_limit_ns = wait_limit_ns();
  CUtensorMap map_a, map_b;
  if (!make_map(&map_a, p.a, p.M, p.K, p.a_stride, (uint32_t)d.q_tile) ||
      !make_map(&map_b, p.b, p.N, p.K, p.b_stride, kP))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(d.tiles < info.sms ? d.tiles : info.sms);
  if (out_dtype == ENGRAM_DTYPE_F32)
    fp8_matmul_kernel<float><<<grid, kThreads, kSmemBytes, stream>>>(map_a, map_b, d);
  else
    fp8_matmul_kernel<uint16_t><<<grid, kThreads, kSmemBytes, stream>>>(map_a, map_b, d);
  return cudaGetLastError();
}

}  // namespace engram

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
// The fp32 accumulator of the tensor cores does not round to nearest: its error grows with
// the number of additions (2e-6 of the result at K = 16,411, against 2.5e-7 of an fp32 sum).
// So K is cut into segments of at most 64 blocks (8192 values) that each start a new
// accumulator, and the epilogue adds the segments in registers, rounding to nearest.
//
// Two persistent kernels walk tiles of out:
//   fp8_matmul_pair_kernel: CTA pairs, tiles of 256 (b) x up to 240 (a) values with
//     tcgen05.mma.cta_group::2 -- each CTA stages its 128 rows of b and half of the rows of
//     a.  240, not 256: two whole accumulators and the scales then fit the 512 columns, and
//     a tile's MMAs follow the last one's without waiting for the epilogue;
//   fp8_matmul_kernel: one CTA per SM, 128 x up to 128 tiles, for products too small to
//     fill the pairs; where even those leave SMs idle (a few rows of a: reading b is the
//     work), 4 or 8 CTAs of a cluster share a tile, each with a part of K, and add their
//     parts through distributed shared memory in rank order; two such CTAs an SM, whose
//     stages together have most of a decode step's weights on the way at once.
// Measured: 65,536 x 4096 x 6144 893 to 937 us by the card (3.5 to 3.7 PFLOP/s; bound by the
// tensor cores, and in a long loop by the power limit: 1100 us near 1.6 GHz); 4096 x 6144 x
// 16,411 with rows 16,416 bytes apart 262 to 277 us (3.0 to 3.2 PFLOP/s; every 128-byte slice of
// a row straddles two lines); few tiles and a long K leave SMs idle: 151 x 5888 x 11,776 27 us
// (its bytes take 11; 46 CTA pairs walk all of K, with 144 and 7 rows of a to a tile, as 4 CTAs
// to a tile would not all be resident), 379 x 2944 x 15,104 25 us (its products take 8.6; 276
// CTAs, 4 to a tile);
// 16 x 4096 x 6144 8.9 us (25 MB of weights, 3.8 us at the copy bandwidth; the rest is the
// launch, the first bytes' latency and the join).
// Warps:
//   0     TMA producer: a ring of stages, each a 128-byte slice along K of the tile's rows
//         of a and b (128-byte swizzle);
//   1     allocates TMEM; one thread (of the pair's even CTA) copies the scales to TMEM
//         (tcgen05.cp) and issues the MMAs into one of two accumulators;
//   2, 3  scales (the pairs' two warps share the work): for every four blocks of K one 32-bit
//         word per row, put into shared memory in the order tcgen05.cp wants (word (r%32)*4 +
//         r/32 of each 128 rows);
//   4..   epilogue: TMEM lanes 32*(warp%4).., stores.
// Every wait is bounded as in wkv_gemm.cu: one that gives up sets ENGRAM_FLAG_TIMEOUT and
// leaves the tiles not yet stored unwritten.
#include <math.h>

#include <mutex>

#include "launch.cuh"
#include "lookup_common.cuh"
#include "tensor_pieces.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr int kP = 128;       // rows of b a tile
constexpr int kQMax = 128;    // most rows of a a tile
constexpr int kThreads = 256;  // warp 3 idles: the epilogue's warps start at a multiple of 4
constexpr int kSegmentBlocks = 64;
constexpr int kScaleSlots = 2;                        // of 16 blocks of K: four groups of four
constexpr uint32_t kGroupBytes = (kP + kQMax) * 4;
constexpr uint32_t kSlotBytes = 4 * kGroupBytes;
constexpr int kMaxStages = 12;
constexpr uint32_t kStageBudget = 192 * 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 2 * kQMax;  // scale words: two buffers of 4 (b) + 4 (a) columns
constexpr size_t kSmemBytes = 1024 + kStageBudget + kScaleSlots * kSlotBytes + 512;
// The CTAs that share a tile's K have one accumulator, half the TMEM and half the shared memory.
constexpr uint32_t kSplitStageBudget = 102 * 1024;
constexpr uint32_t kSplitTmemCols = 256, kSplitScaleCol = kQMax;
constexpr size_t kSplitSmemBytes = 1024 + kSplitStageBudget + kScaleSlots * kSlotBytes + 512;
static_assert(2 * (kSplitSmemBytes + 1024 + 64) <= 228 * 1024);

struct MatmulDev {
  const uint8_t *a_scale, *b_scale;
  void *out;
  int32_t *status;
  int64_t M, N, out_stride;
  int32_t kblocks, a_shift, b_shift;  // log2 of the rows sharing a scale (0 or 7)
  int32_t q_tile, stages;
  int32_t segments, seg_blocks;  // K in segments of seg_blocks blocks (a multiple of 4)
  int32_t splits;                // CTAs that share a tile's K (a cluster)
  int64_t tiles_p, tiles_q, tiles;
  int64_t wait_limit_ns;
  bool withhold;  // test hook: the first stage waits for bytes that never come
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

// The whole warp waits; the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                          const MatmulDev &p) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p.wait_limit_ns, p.status));
}

// The scale bytes of 16 blocks of K (from block kb on, a multiple of 16) of one row, as whole
// aligned words and the shift to their first byte, so that they can be in flight while the
// batch before them is written.  Bytes past the last block are whatever follows (no MMA reads
// them), rows past the last one zero; single bytes are loaded only where a word would reach
// outside the array.
struct Scales {
  uint32_t v[5], shift;

  __device__ __forceinline__ void load(const uint8_t *s, int64_t row, int64_t rows, int row_shift, int kb,
                                       int kblocks) {
    shift = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = 0;
    if (row >= rows) return;
    const uint8_t *end = s + (((rows - 1) >> row_shift) + 1) * kblocks;
    const uint8_t *src = s + (row >> row_shift) * kblocks + kb;
    const uint32_t off = (uint32_t)((uintptr_t)src & 3);
    const uint8_t *word = src - off;
    if (word >= s && word + 20 <= end) {
      shift = 8 * off;
#pragma unroll
      for (int i = 0; i < 5; ++i) v[i] = __ldg(reinterpret_cast<const uint32_t *>(word) + i);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (kb + i < kblocks) v[i >> 2] |= (uint32_t)__ldg(src + i) << (8 * (i & 3));
    }
  }
  // The bytes of blocks kb + 4g .. kb + 4g + 3.
  __device__ __forceinline__ uint32_t word(int g) const { return __funnelshift_r(v[g], v[g + 1], shift); }
};

// Tiles in groups of up to 16 along b, a's tiles inside a group in order: what the resident
// CTAs read at one time is a few slices of each operand.
__device__ __forceinline__ void tile_at(const MatmulDev &p, int64_t tile, int64_t &tp, int64_t &tq) {
  const int64_t per = 16 * p.tiles_q, g = tile / per, in = tile - g * per;
  const int64_t wide = min((int64_t)16, p.tiles_p - g * 16);
  tq = in / wide;
  tp = g * 16 + in - tq * wide;
}

template <typename TO>
__device__ __forceinline__ void store_out(TO *dst, uint32_t v) {
  if constexpr (sizeof(TO) == 4)
    *dst = __uint_as_float(v);
  else
    *dst = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v)));
}

// A warp's part of an accumulator -- 32 lanes (outputs n, n + 1, ..), `chunks` times 16 columns
// (outputs m0, m0 + 1, ..) -- goes to memory or (MULTI) into sums over the segments that the
// last one stores.  `release` runs once the last column is in registers, before its stores.
// The sums move through the registers so that one chunk's code serves all: written out per
// chunk it was fetched once a tile, from beyond the instruction cache, and that took 13 us of
// 47 for one tile of 92 blocks (151 x 5888 x 11,776).
template <typename TO, int CHUNKS, bool MULTI>
struct Drain {
  float sum[MULTI ? CHUNKS * 16 : 1];

  template <typename F>
  __device__ __forceinline__ void run(uint32_t taddr, int chunks, bool first, bool last, TO *out, int64_t stride,
                                      int64_t m0, int64_t M, bool mine, F release) {
    const int rows = (int)min((int64_t)chunks * 16, M - m0);
    if constexpr (MULTI) {
      out += m0 * stride;
#pragma unroll 1
      for (int c = 0; c < CHUNKS; ++c) {
        uint32_t v[16];
        __syncwarp();  // together again after the stores, as tcgen05.ld wants the warp
        if (c < chunks) tmem_ld16(taddr + c * 16, v);
        if (c == chunks - 1) release();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (!first) v[i] = __float_as_uint(sum[i] + __uint_as_float(v[i]));
          if (last && mine && c * 16 + i < rows) store_out(out, v[i]);
          out += stride;
        }
        // The chunk's sums go to the back: after CHUNKS turns each is in its place again.
#pragma unroll
        for (int i = 0; i < CHUNKS * 16 - 16; ++i) sum[i] = sum[i + 16];
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[CHUNKS * 16 - 16 + i] = __uint_as_float(v[i]);
      }
    } else {
      out += m0 * stride;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint32_t v[16];
        __syncwarp();  // as above
        tmem_ld16(taddr + c * 16, v);
        if (c == chunks - 1) release();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (mine && c * 16 + i < rows) store_out(out, v[i]);
          out += stride;
        }
      }
    }
  }
};

template <typename TO, bool MULTI, bool SPLIT>
__global__ void __launch_bounds__(kThreads, SPLIT ? 2 : 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ MatmulDev p) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t *slots = sm + (SPLIT ? kSplitStageBudget : kStageBudget);
  constexpr uint32_t kCols = SPLIT ? kSplitTmemCols : kTmemCols;
  constexpr uint32_t kScales = SPLIT ? kSplitScaleCol : kScaleCol;
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
  const int stages = p.stages, qt = p.q_tile;
  const uint32_t stage_bytes = (uint32_t)(kP + qt) * 128;
  // This CTA's blocks of K (from kb_first on) and its tiles.
  const int rank = SPLIT ? (int)cluster_rank() : 0;
  const int kb_first = SPLIT ? p.kblocks * rank / p.splits : 0;
  const int kblocks = SPLIT ? p.kblocks * (rank + 1) / p.splits - kb_first : p.kblocks;
  const int64_t first_tile = SPLIT ? blockIdx.x / p.splits : blockIdx.x;
  const int64_t tile_step = SPLIT ? gridDim.x / p.splits : gridDim.x;

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
    if (p.withhold) mbar_expect_tx(full, 16);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- TMA producer
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
        int64_t tp, tq;
        tile_at(p, tile, tp, tq);
        const int p0 = (int)(tp * kP), q0 = (int)(tq * qt);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          if (!(ok = wait_phase(empty + s, ph ^ 1, abort_flag, p.wait_limit_ns, p.status))) break;
          uint8_t *st = sm + s * stage_bytes;
          mbar_arrive_expect_tx(full + s, stage_bytes);
          tma_load_2d(st, &map_b, (kb_first + kb) * 128, p0, full + s);
          tma_load_2d(st + kP * 128, &map_a, (kb_first + kb) * 128, q0, full + s);
          if (++s == stages) s = 0, ph ^= 1;
        }
      }
      // Loads issued into shared memory land before the block can exit.
      for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j)
        drain_phase(full + j % stages, (j / stages) & 1, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The warp runs the loop together, so that what the instructions take (descriptors,
    // columns) is computed once in its uniform registers; one lane issues.
    uint32_t unit = 0, batch = 0;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const bool one = elect_one();
    for (int64_t tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
      for (int kb0 = 0; ok && kb0 < kblocks; kb0 += p.seg_blocks, ++unit) {
        const int kb1 = min(kb0 + p.seg_blocks, kblocks);
        const uint32_t acc = unit & 1, use = unit >> 1;
        if (!(ok = warp_wait(acc_empty + acc, (use & 1) ^ 1, abort_flag, p))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + acc * kQMax;
        uint32_t sp = 0, sq = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
          if ((kb & 3) == 0) {  // the scales of the next four blocks
            const int slot = batch & 1;
            if ((kb & 15) == 0) {
              if (!(ok = warp_wait(sc_full + slot, (batch >> 1) & 1, abort_flag, p))) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            sp = tmem + kScales + (kb >> 2 & 1) * 8, sq = sp + 4;
            const uint64_t src =
                smem_desc_scales(smem_u32(slots + slot * kSlotBytes + (kb >> 2 & 3) * kGroupBytes));
            const bool done = (kb & 15) == 12 || kb + 4 >= kblocks;  // with this slot
            if (one) {
              copy_scales(sp, src);
              copy_scales(sq, src + (kP * 4 >> 4));
              if (done) umma_commit(sc_empty + slot);
            }
            batch += done;
          }
          if (!(ok = warp_wait(full + s, ph, abort_flag, p))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t ps = smem_u32(sm + s * stage_bytes);
          const uint64_t pd = smem_desc_sw128(ps), qd = smem_desc_sw128(ps + kP * 128);
          const uint32_t idesc = instr_desc(kP, qt, kb & 3);
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 values along K: 32 bytes
              umma_fp8(d, pd + 2 * k, qd + 2 * k, idesc, sp, sq, kb != kb0 || k != 0 ? 1u : 0u);
            umma_commit(empty + s);
          }
          __syncwarp();
          if (++s == stages) s = 0, ph ^= 1;
        }
        if (ok && one) umma_commit(acc_full + acc);
        __syncwarp();
      }
    }
    if (one) umma_commit(mma_done);
    __syncwarp();
  } else if (warp == 2) {
    // --------------------------------------------------------------- scales
    // 16 blocks of K at a time, the next batch's loads in flight under this one's waits.
    uint32_t batch = 0;
    bool ok = true;
    const auto load = [&](int64_t tile, int kb, Scales(&w)[8]) {
      if (tile >= p.tiles) return;
      int64_t p0, q0;
      tile_at(p, tile, p0, q0);
      p0 *= kP, q0 *= qt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i].load(p.b_scale, p0 + 32 * i + lane, p.N, p.b_shift, kb_first + kb, p.kblocks);
        w[4 + i].load(p.a_scale, q0 + 32 * i + lane, 32 * i < qt ? p.M : 0, p.a_shift, kb_first + kb,
                      p.kblocks);
      }
    };
    Scales w[8];
    int64_t tile = first_tile;
    int kb = 0;
    load(tile, kb, w);
    while (ok && tile < p.tiles) {
      const int64_t next_tile = kb + 16 < kblocks ? tile : tile + tile_step;
      const int next_kb = kb + 16 < kblocks ? kb + 16 : 0;
      Scales next[8];
      load(next_tile, next_kb, next);
      const int slot = batch & 1;
      if (!(ok = warp_wait(sc_empty + slot, ((batch >> 1) & 1) ^ 1, abort_flag, p))) break;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint4 *dst = reinterpret_cast<uint4 *>(slots + slot * kSlotBytes + g * kGroupBytes);
        dst[lane] = make_uint4(w[0].word(g), w[1].word(g), w[2].word(g), w[3].word(g));
        dst[32 + lane] = make_uint4(w[4].word(g), w[5].word(g), w[6].word(g), w[7].word(g));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_full + slot);
      ++batch;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = next[i];
      tile = next_tile, kb = next_kb;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    uint32_t unit = 0;
    bool ok = true;
    Drain<TO, kQMax / 16, MULTI> drain;
    for (int64_t tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
      int64_t tp, tq;
      tile_at(p, tile, tp, tq);
      const int64_t n = tp * kP + quad * 32 + lane, m0 = tq * qt;
      TO *out = static_cast<TO *>(p.out) + n;
      for (int seg = 0; seg < p.segments; ++seg, ++unit) {
        const uint32_t acc = unit & 1, use = unit >> 1;
        ok = warp_wait(acc_full + acc, use & 1, abort_flag, p);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + acc * kQMax;
        if constexpr (SPLIT) {
          // The partial tile into shared memory (the stages: every MMA has read them).
          float *part = reinterpret_cast<float *>(sm) + quad * 32 + lane;
          for (int c = 0; c < qt; c += 16) {
            uint32_t v[16];
            tmem_ld16(base + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * kP] = __uint_as_float(v[i]);
          }
          break;
        }
        drain.run(base, qt / 16, seg == 0, seg == p.segments - 1, out, p.out_stride, m0, p.M, n < p.N, [&] {
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + acc);
        });
      }
    }
  }

  if constexpr (SPLIT) {
    // Each CTA adds a share of the tile's columns over the cluster, in rank order.
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();
    bool ok = true;
    for (int r = 0; r < p.splits; ++r)  // a CTA that gave up has no partial tile
      ok &= load_cluster(map_to_rank(smem_u32(const_cast<int *>(abort_flag)), r)) == 0;
    int64_t tp, tq;
    tile_at(p, first_tile, tp, tq);
    // A warp a column (128 outputs of one row of out), four outputs a lane.
    const int64_t n = tp * kP + lane * 4;
    const int q_end = qt * (rank + 1) / p.splits;
    for (int q = qt * rank / p.splits + warp; q < q_end; q += kThreads / 32) {
      const int64_t m = tq * qt + q;
      const uint32_t at = smem_u32(sm) + (q * kP + lane * 4) * 4;
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = r < p.splits ? load4_cluster(map_to_rank(at, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 1; r < 8; ++r)
        v[0].x += v[r].x, v[0].y += v[r].y, v[0].z += v[r].z, v[0].w += v[r].w;
      const float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      TO *out = static_cast<TO *>(p.out) + m * p.out_stride + n;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ok && n + i < p.N && m < p.M) store_out(out + i, __float_as_uint(sum[i]));
    }
    cluster_sync();  // no CTA leaves while another may still read its part
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) drain_phase(mma_done, 0, p.wait_limit_ns);
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                 : "memory");
  }
}

// ---- CTA pairs ------------------------------------------------------------------------

constexpr int kPairQMax = 240;
constexpr int kPairThreads = 512;
constexpr int kPairParts = 3;  // of a tile's columns, a warp of each quarter of the lanes each
constexpr uint32_t kPairStageBudget = 213 * 1024;
constexpr uint32_t kPairGroupBytes = (kP + 256) * 4;
constexpr uint32_t kPairSlotBytes = 4 * kPairGroupBytes;
constexpr uint32_t kPairScaleCol = 2 * kPairQMax;  // scale words: two buffers of 4 (b) + 8 (a) columns
constexpr size_t kPairSmemBytes = 1024 + kPairStageBudget + kScaleSlots * kPairSlotBytes + 512;
static_assert(kPairScaleCol + 2 * 12 <= kTmemCols && kPairSmemBytes <= 227 * 1024);

__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void umma_fp8_pair(uint32_t d, uint64_t p_desc, uint64_t q_desc, uint32_t idesc,
                                              uint32_t sp, uint32_t sq, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(p_desc), "l"(q_desc), "r"(idesc), "r"(sp), "r"(sq), "r"(accumulate)
      : "memory");
}

// Barriers as in wkv_gemm_pair_kernel: full and sc_full live in the leader (the even CTA),
// sc_full with one arrival per scale warp; empty, sc_empty, acc_full and mma_done exist
// in both and take the leader's multicast commits; acc_empty lives in the leader and takes an
// arrival from every epilogue warp of the pair.
template <typename TO, bool MULTI>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                           const __grid_constant__ CUtensorMap map_b, const __grid_constant__ MatmulDev p) {
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks = p.kblocks, stages = p.stages, qt = p.q_tile;
  const uint32_t stage_bytes = (uint32_t)(kP + qt / 2) * 128;
  uint8_t *slots = sm + kPairStageBudget;
  uint64_t *full = reinterpret_cast<uint64_t *>(slots + kScaleSlots * kPairSlotBytes);
  uint64_t *empty = full + kMaxStages;
  uint64_t *sc_full = empty + kMaxStages;
  uint64_t *sc_empty = sc_full + kScaleSlots;
  uint64_t *acc_full = sc_empty + kScaleSlots;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const uint32_t rank = cluster_rank();
  const int64_t cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(sc_full + s, 4);
      mbar_init(sc_empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full + a, 1);
      mbar_init(acc_empty + a, 2 * 4 * kPairParts);
    }
    mbar_init(mma_done, 1);
    if (p.withhold) mbar_expect_tx(full, 16);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();  // both CTAs' barriers are initialised before either uses the other's
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      // ----------------------------------------------- TMA producer (both CTAs)
      const uint32_t full_lead = map_to_rank(smem_u32(full), 0);
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t tile = cluster; ok && tile < p.tiles; tile += n_clusters) {
        int64_t tp, tq;
        tile_at(p, tile, tp, tq);
        const int p0 = (int)(tp * 2 * kP) + (int)rank * kP, q0 = (int)(tq * qt) + (int)rank * (qt / 2);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          if (!(ok = wait_phase(empty + s, ph ^ 1, abort_flag, p.wait_limit_ns, p.status))) break;
          uint8_t *st = sm + s * stage_bytes;
          const uint32_t bar = full_lead + 8u * s;
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * stage_bytes);
          tma_load_2d_pair(st, &map_b, kb * 128, p0, bar);
          tma_load_2d_pair(st + kP * 128, &map_a, kb * 128, q0, bar);
          if (++s == stages) s = 0, ph ^= 1;
        }
      }
      // The leader's full barriers count both CTAs' bytes.
      if (rank == 0)
        for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j)
          drain_phase(full + j % stages, (j / stages) & 1, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------- MMA issuer (leader)
      uint32_t unit = 0, batch = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const bool one = elect_one();
      for (int64_t tile = cluster; ok && tile < p.tiles; tile += n_clusters) {
        for (int kb0 = 0; ok && kb0 < kblocks; kb0 += p.seg_blocks, ++unit) {
          const int kb1 = min(kb0 + p.seg_blocks, kblocks);
          const uint32_t acc = unit & 1, use = unit >> 1;
          if (!(ok = warp_wait(acc_empty + acc, (use & 1) ^ 1, abort_flag, p))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t d = tmem + acc * kPairQMax;
          uint32_t sp = 0, sq = 0;
          for (int kb = kb0; kb < kb1; ++kb) {
            if ((kb & 3) == 0) {
              const int slot = batch & 1;
              // Both CTAs' words: their writers fenced them for the async proxy and released
              // them to the cluster.  This thread does not read them (tcgen05.cp does), so a
              // cluster-scope acquire is not needed.
              if ((kb & 15) == 0) {
                if (!(ok = warp_wait(sc_full + slot, (batch >> 1) & 1, abort_flag, p))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              }
              sp = tmem + kPairScaleCol + (kb >> 2 & 1) * 12, sq = sp + 4;
              const uint64_t src =
                  smem_desc_scales(smem_u32(slots + slot * kPairSlotBytes + (kb >> 2 & 3) * kPairGroupBytes));
              const bool done = (kb & 15) == 12 || kb + 4 >= kblocks;
              if (one) {
                copy_scales_pair(sp, src);
                copy_scales_pair(sq, src + (kP * 4 >> 4));
                if (qt > 128) copy_scales_pair(sq + 4, src + (2 * kP * 4 >> 4));
                if (done) umma_commit_pair(sc_empty + slot);
              }
              batch += done;
            }
            if (!(ok = warp_wait(full + s, ph, abort_flag, p))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t ps = smem_u32(sm + s * stage_bytes);
            const uint64_t pd = smem_desc_sw128(ps), qd = smem_desc_sw128(ps + kP * 128);
            const uint32_t idesc = instr_desc(2 * kP, qt, kb & 3);
            if (one) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_fp8_pair(d, pd + 2 * k, qd + 2 * k, idesc, sp, sq, kb != kb0 || k != 0 ? 1u : 0u);
              umma_commit_pair(empty + s);
            }
            __syncwarp();
            if (++s == stages) s = 0, ph ^= 1;
          }
          if (ok && one) umma_commit_pair(acc_full + acc);
          __syncwarp();
        }
      }
      if (one) umma_commit_pair(mma_done);
      __syncwarp();
    }
  } else if (warp < 4) {
    // --------------------------- scales (both CTAs: own rows of b, all rows of a)
    // 12 rows a lane: warp 2 takes the four of b and two of a, warp 3 six of a; 16 blocks of
    // K at a time, the next batch's loads in flight under this one's waits.
    const uint32_t sc_full_lead = map_to_rank(smem_u32(sc_full), 0);
    const bool first = warp == 2;
    uint32_t batch = 0;
    bool ok = true;
    const auto load = [&](int64_t tile, int kb, Scales(&w)[6]) {
      if (tile >= p.tiles) return;
      int64_t p0, q0;
      tile_at(p, tile, p0, q0);
      p0 = p0 * 2 * kP + rank * kP, q0 *= qt;
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        const int r = first ? i : 6 + i;  // of the 12
        if (r < 4)
          w[i].load(p.b_scale, p0 + 32 * r + lane, p.N, p.b_shift, kb, kblocks);
        else
          w[i].load(p.a_scale, q0 + 32 * (r - 4) + lane, 32 * (r - 4) < qt ? p.M : 0, p.a_shift, kb, kblocks);
      }
    };
    Scales w[6];
    int64_t tile = cluster, next_tile = cluster;
    int kb = kblocks, next_kb = 0;
    while (ok) {
      Scales next[6];
      load(next_tile, next_kb, next);
      if (kb < kblocks) {  // not the first time
        const int slot = batch & 1;
        if (!(ok = warp_wait(sc_empty + slot, ((batch >> 1) & 1) ^ 1, abort_flag, p))) break;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t *dst =
              reinterpret_cast<uint32_t *>(slots + slot * kPairSlotBytes + g * kPairGroupBytes) + lane * 4;
          if (first) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0].word(g), w[1].word(g), w[2].word(g), w[3].word(g));
            *reinterpret_cast<uint2 *>(dst + 128) = make_uint2(w[4].word(g), w[5].word(g));
          } else {
            *reinterpret_cast<uint2 *>(dst + 130) = make_uint2(w[0].word(g), w[1].word(g));
            *reinterpret_cast<uint4 *>(dst + 256) =
                make_uint4(w[2].word(g), w[3].word(g), w[4].word(g), w[5].word(g));
          }
        }
        // Once for 16 blocks: the fence and the cluster-wide release wait for everything this
        // warp has in flight, and once for four blocks they took longer than the blocks.
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(sc_full_lead + 8u * slot);
        ++batch;
      }
      if ((tile = next_tile) >= p.tiles) break;
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = next[i];
      kb = next_kb;
      next_kb = kb + 16 < kblocks ? kb + 16 : 0;
      next_tile = next_kb ? tile : tile + n_clusters;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const uint32_t acc_empty_lead = map_to_rank(smem_u32(acc_empty), 0);
    // This warp's 16-column chunks: a part of the tile's.
    const int c0 = qt / 16 * part / kPairParts, chunks = qt / 16 * (part + 1) / kPairParts - c0;
    uint32_t unit = 0;
    bool ok = true;
    Drain<TO, (kPairQMax / 16 + kPairParts - 1) / kPairParts, MULTI> drain;
    for (int64_t tile = cluster; ok && tile < p.tiles; tile += n_clusters) {
      int64_t tp, tq;
      tile_at(p, tile, tp, tq);
      const int64_t n = tp * 2 * kP + rank * kP + quad * 32 + lane, m0 = tq * qt + c0 * 16;
      TO *out = static_cast<TO *>(p.out) + n;
      for (int seg = 0; seg < p.segments; ++seg, ++unit) {
        const uint32_t acc = unit & 1, use = unit >> 1;
        ok = warp_wait(acc_full + acc, use & 1, abort_flag, p);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + acc * kPairQMax + c0 * 16;
        drain.run(base, chunks, seg == 0, seg == p.segments - 1, out, p.out_stride, m0, p.M, n < p.N, [&] {
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_lead + 8u * acc);
        });
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1 && lane == 0) drain_phase(mma_done, 0, p.wait_limit_ns);  // the pair's MMAs ran
  __syncwarp();
  cluster_sync();  // no CTA leaves while the other may still signal it
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
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
  int sms = 0, pairs = 0;  // pairs: CTA pairs that fit at once
};
DeviceInfo g_info[64];
std::mutex g_info_mu;

using Kernel = void (*)(CUtensorMap, CUtensorMap, MatmulDev);
enum Form { kSingle, kSingleMulti, kSplit, kPair, kPairMulti, kForms };
Kernel kernel_of(int form, bool f32) {
  static constexpr Kernel all[kForms][2] = {
      {fp8_matmul_kernel<uint16_t, false, false>, fp8_matmul_kernel<float, false, false>},
      {fp8_matmul_kernel<uint16_t, true, false>, fp8_matmul_kernel<float, true, false>},
      {fp8_matmul_kernel<uint16_t, false, true>, fp8_matmul_kernel<float, false, true>},
      {fp8_matmul_pair_kernel<uint16_t, false>, fp8_matmul_pair_kernel<float, false>},
      {fp8_matmul_pair_kernel<uint16_t, true>, fp8_matmul_pair_kernel<float, true>}};
  return all[form][f32];
}

cudaError_t device_info(DeviceInfo &out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_info_mu);
  DeviceInfo &d = g_info[dev & 63];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i = 0; i < 2 * kForms && e == cudaSuccess; ++i)
      e = cudaFuncSetAttribute(kernel_of(i / 2, i & 1), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(i / 2 >= kPair ? kPairSmemBytes : i / 2 == kSplit ? kSplitSmemBytes : kSmemBytes));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(d.sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kPairSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&d.pairs, kernel_of(kPair, true), &cfg)) != cudaSuccess) return e;
    d.ready = true;
  }
  out = d;
  return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
  d.wait_limit_ns = wait_limit_ns();
  d.withhold = take_withheld_launch();
  const int64_t segments = ceil_div(d.kblocks, kSegmentBlocks);
  d.seg_blocks = (int32_t)(ceil_div(ceil_div(d.kblocks, segments), 4) * 4);
  d.segments = (int32_t)ceil_div(d.kblocks, d.seg_blocks);
  // The form and the width of a tile along a go by an estimate of their time in microseconds,
  // less the launch's, fitted to all forms over M 1 .. 16,384, N 128 .. 8192, K 256 .. 16,384:
  //   single: 1.3 + 0.23 a block of K, for each wave of tiles over the SMs;
  //   pairs:  2.1 + max(0.2, 0.00118 (width + 16)) a block, but at least what draining the
  //           tile takes, 4.6 at 240 columns; for each wave over the pairs, and 1.5 once;
  //   split:  4 or 8 CTAs share a tile's K where there is room for them, two an SM: 0.25 a
  //           block of a CTA's part, and the joining, 2.4 + 0.02 a column of the tile and
  //           0.00014 a column of each CTA.
  // (16 x 4096 x 6144: split in 8 9.0 us, single 14.2; 512 x 1024 x 8192: in 4 13.3, in 8 14.5,
  // single 18.5, pairs 19.1; 16 x 4096 x 1024: in 8 6.4, single 5.4.)
  const double kb = d.kblocks;
  const int q_single = (int)(p.M < kQMax ? ceil_div(p.M, 16) * 16 : kQMax);
  const int64_t single_tiles = ceil_div(p.N, kP) * ceil_div(p.M, q_single);
  const double single_us = ceil_div(single_tiles, info.sms) * (1.3 + 0.23 * kb);
  double pair_us = HUGE_VAL;
  if (info.pairs > 0 && p.M > 128 && p.N > 128) {
    for (int qt = kPairQMax; qt >= 128; qt -= 16) {
      const int64_t waves = ceil_div(ceil_div(p.N, 2 * kP) * ceil_div(p.M, qt), info.pairs);
      const double block = fmax(0.2, 0.00118 * (qt + 16));
      const double us = 1.5 + waves * fmax(4.6 * qt / kPairQMax, 2.1 + block * kb);
      if (us < pair_us) pair_us = us, d.q_tile = qt;
    }
  }
  double split_us = HUGE_VAL;
  for (int n = 4; n <= 8; n *= 2) {
    if (n * single_tiles > 2 * info.sms || d.kblocks < n || ceil_div(d.kblocks, n) > kSegmentBlocks) continue;
    const double us = 0.25 * kb / n + 2.4 + 0.02 * q_single + 0.00014 * q_single * n * single_tiles;
    if (us < split_us) split_us = us, d.splits = n;
  }
  const bool split = split_us < single_us && split_us < pair_us, pair = !split && pair_us < single_us;
  int form;
  if (pair) {
    form = d.segments > 1 ? kPairMulti : kPair;
    d.tiles_p = ceil_div(p.N, 2 * kP);
    d.stages = (int32_t)(kPairStageBudget / ((kP + d.q_tile / 2) * 128));
  } else {
    form = split ? kSplit : d.segments > 1 ? kSingleMulti : kSingle;
    d.tiles_p = ceil_div(p.N, kP);
    d.q_tile = q_single;
    d.stages = (int32_t)((split ? kSplitStageBudget : kStageBudget) / ((kP + d.q_tile) * 128));
    if (split) {  // a CTA's part of K is one segment
      d.segments = 1;
      d.seg_blocks = kSegmentBlocks;
    }
  }
  if (d.stages > kMaxStages) d.stages = kMaxStages;
  d.tiles_q = ceil_div(p.M, d.q_tile);
  d.tiles = d.tiles_p * d.tiles_q;
  CUtensorMap map_a, map_b;
  if (!make_map(&map_a, p.a, p.M, p.K, p.a_stride, (uint32_t)(pair ? d.q_tile / 2 : d.q_tile)) ||
      !make_map(&map_b, p.b, p.N, p.K, p.b_stride, kP))
    return cudaErrorInvalidValue;
  const Kernel kernel = kernel_of(form, out_dtype == ENGRAM_DTYPE_F32);
  if (pair)
    return launch(kernel, 2 * (d.tiles < info.pairs ? d.tiles : info.pairs), kPairThreads, kPairSmemBytes,
                  stream, 2, map_a, map_b, d);
  if (form == kSplit)
    return launch(kernel, d.tiles * d.splits, kThreads, kSplitSmemBytes, stream, d.splits, map_a, map_b, d);
  return launch(kernel, d.tiles < info.sms ? d.tiles : info.sms, kThreads, kSmemBytes, stream, 1, map_a,
                map_b, d);
}

}  // namespace engram

// product.cu -- out = act(scale * a b^T + bias) + residual for 16-bit operands, on the sm_103a
// tensor cores (tcgen05.mma kind::f16, fp32 accumulators in TMEM).
//
// The roles are turned around: the rows of b (the output's columns) are the instruction's M
// rows, the rows of a its N columns, so that a warp of the epilogue holds 32 neighbouring
// outputs of one row of out in its lanes and reads and stores whole lines for any stride and
// size.  Either operand may run along K in memory (K-major) or along its rows (MN-major: boxes
// of 64 rows x 64 of K, told to the instruction by its descriptors), so the gradient's products
// and those of the symmetric iteration need no transposed copies.
//
// Two persistent kernels walk tiles of out:
//   pairs: CTA pairs (tcgen05.mma.cta_group::2), tiles of 256 (b) x up to 256 (a) values -- each
//     CTA stages its 128 rows of b and half of the rows of a;
//   single: one CTA, 128 x up to 128 tiles, for products too small to fill the pairs; where even
//     those leave SMs idle (a few rows of a: reading b is the work), 4 or 8 CTAs of a cluster
//     share a tile, each with a part of K, and add their parts through distributed shared memory
//     in rank order, two such CTAs an SM.
// Warps: 0 TMA producer (a ring of stages of 64 of K, 128-byte swizzle); 1 allocates TMEM, one
// thread (of the pair's even CTA) issues the MMAs into one of two accumulators; 4.. epilogue.
//
// The fp32 accumulator of the tensor cores does not round to nearest: its error grows with the
// number of additions.  For fp32 outputs K is cut into segments of at most 8192 that each start
// a new accumulator, and the epilogue adds them to the sum so far, which it keeps in out,
// rounding to nearest.
//
// A symmetric product (both operands one matrix) computes the tiles on one side of the diagonal
// and stores every value twice, the second time transposed: a lane's 16 values of a chunk are
// neighbours there.
//
// Every wait is bounded as in wkv_gemm.cu: one that gives up sets ENGRAM_FLAG_TIMEOUT and leaves
// the tiles not yet stored unwritten.
#include <math.h>

#include <mutex>

#include "launch.cuh"
#include "product_internal.cuh"
#include "tensor_core.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kP = 128;         // rows of b a CTA stages
constexpr int kBK = 64;         // of K a stage: 128 bytes
constexpr int kQMax = 128;      // most rows of a a tile of one CTA
constexpr int kPairQMax = 256;  // and of a pair
constexpr int kThreads = 256;   // warps 2 and 3 idle: the epilogue's start at a multiple of 4
constexpr int kPairThreads = 512;
constexpr int kPairParts = 3;  // of a tile's columns, a warp of each quarter of the lanes each
constexpr int kSegmentBlocks = 128;
constexpr int kMaxStages = 12;
constexpr uint32_t kPBytes = kP * kBK * 2;
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kStageBudget = 192 * 1024;
constexpr uint32_t kSplitStageBudget = 104 * 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSplitTmemCols = 128;
constexpr size_t kSmemBytes = 1024 + kStageBudget + kBarBytes;
constexpr size_t kSplitSmemBytes = 1024 + kSplitStageBudget + kBarBytes;
constexpr uint32_t kPairStageBudget = 224 * 1024;
constexpr size_t kPairSmemBytes = 1024 + kPairStageBudget + kBarBytes;
static_assert(2 * (kSplitSmemBytes + 1024 + 64) <= 228 * 1024 && kPairSmemBytes <= 227 * 1024);
static_assert((2 * kMaxStages + 6) * 8 + 8 <= kBarBytes);

struct ProductDev {
  Plane out, residual, pre;
  const void *bias;
  int32_t *status;
  int64_t wait_limit_ns;
  int32_t M, N;
  float scale, residual_scale;
  int32_t bias_type, act;
  int32_t kblocks, q_tile, q_rows, stages;  // q_rows: rows of a that a CTA stages
  int32_t segments, seg_blocks, splits;
  int32_t tiles_p, tiles_q, tiles, matrix_tiles;
  uint32_t idesc;
  bool p_t, q_t, symmetric, many;
  bool fold;      // the residual goes into the first segment's sum (it lies where out does)
  bool withhold;  // test hook: the first stage waits for bytes that never come
};

// Shared-memory descriptor of an operand tile, 128-byte swizzle.  K-major: rows of 64 of K,
// 8-row groups 1024 bytes apart.  MN-major: boxes of 64 rows (128 bytes) by 64 of K, 8192 bytes
// apart along the rows, groups of 8 along K 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool t) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(t ? 8192 >> 4 : 1) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// What 16 of K add to it, in its units of 16 bytes.
__device__ __forceinline__ uint32_t desc_step(bool t) { return t ? 2048 >> 4 : 32 >> 4; }

template <bool PAIR>
__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t p_desc, uint64_t q_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(p_desc), "l"(q_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(p_desc), "l"(q_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (PAIR)
    umma_commit_pair(bar);
  else
    umma_commit(bar);
}

// 3-D TMA load of this CTA completing on `bar`: a shared::cta address, or with PAIR a
// shared::cluster one, of either CTA of the pair.
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The rows from r0 on of one operand, 64 of K from k on, into a stage.
template <bool PAIR>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, bool t, int r0, int rows,
                                             int k, int z, uint32_t bar) {
  if (t) {
    for (int r = 0; r < rows; r += 64) tma_load_3d<PAIR>(dst + r * 128, map, r0 + r, k, z, bar);
  } else {
    tma_load_3d<PAIR>(dst, map, k, r0, z, bar);
  }
}

// The whole warp waits; the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                          const ProductDev &p) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p.wait_limit_ns, p.status));
}

struct Tile {
  int p0, q0, z;
};
// Tiles in groups of up to 16 along b, a's tiles inside a group in order: what the resident
// CTAs read at one time is a few slices of each operand.  Of a symmetric product those that
// hold any output (m, n) with n <= m.
template <int WIDTH>
__device__ __forceinline__ Tile tile_at(const ProductDev &p, int tile) {
  Tile r{0, 0, 0};
  uint32_t t = tile;
  if (p.many) {
    r.z = t / (uint32_t)p.matrix_tiles;
    t -= r.z * (uint32_t)p.matrix_tiles;
  }
  uint32_t tp, tq;
  if (p.symmetric) {
    for (tq = 0;; ++tq) {
      const uint32_t wide = min(p.tiles_p, (min(p.M, (int)(tq + 1) * p.q_tile) - 1) / WIDTH + 1);
      if (t < wide) break;
      t -= wide;
    }
    tp = t;
  } else {
    const uint32_t per = 16u * p.tiles_q, g = t / per, in = t - g * per;
    const uint32_t wide = min(16u, p.tiles_p - g * 16u);
    tq = in / wide;
    tp = g * 16 + in - tq * wide;
  }
  r.p0 = (int)tp * WIDTH, r.q0 = (int)tq * p.q_tile;
  return r;
}

// ---- epilogue ---------------------------------------------------------------------------

// f(a null pointer of the C++ type of `type`).
template <typename F>
__device__ __forceinline__ void by_type(int type, F f) {
  if (type == ENGRAM_DTYPE_F32)
    f(static_cast<float *>(nullptr));
  else if (type == ENGRAM_DTYPE_BF16)
    f(static_cast<__nv_bfloat16 *>(nullptr));
  else
    f(static_cast<__half *>(nullptr));
}

template <int N>
__device__ __forceinline__ void activate(float (&x)[N], int act) {
  if (act == ENGRAM_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] < 0.f ? 0.f : x[i];  // a NaN stays
  } else if (act == ENGRAM_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __fdividef(x[i], 1.f + __expf(-x[i]));
  } else if (act == ENGRAM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.5f * x[i] * (1.f + erff(x[i] * 0.70710678f));
  }
}

// N values of one column of out (x[i] is output (m0 + i, n)), or of one row (ROW: (m, n0 + i)),
// of which the first `count` count.
template <bool ROW, int N>
__device__ __forceinline__ void load_values(const Plane &s, int64_t z, int64_t m, int64_t n, int count,
                                            float (&x)[N]) {
  by_type(s.type, [&](auto *type) {
    auto *src = static_cast<decltype(type)>(s.p) + z * s.batch + m * s.stride + n;
    const int64_t step = ROW ? 1 : s.stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = i < count ? to_float(*src) : 0.f;
      src += step;
    }
  });
}
template <bool ROW, int N>
__device__ __forceinline__ void store_values(const Plane &d, int64_t z, int64_t m, int64_t n, int count,
                                             const float (&x)[N]) {
  by_type(d.type, [&](auto *type) {
    auto *dst = static_cast<decltype(type)>(d.p) + z * d.batch + m * d.stride + n;
    const int64_t step = ROW ? 1 : d.stride;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < count) from_float(*dst, x[i]);
      dst += step;
    }
  });
}

// Sums of products become outputs: (m + i, n), or with ROW (m, n + i), for i < count.
// `loaded`: the residual's values, already on their way.
template <bool ROW, int N>
__device__ __forceinline__ void finish(const ProductDev &p, int64_t z, int64_t m, int64_t n, int count, bool first,
                                       bool last, float (&x)[N], const float (&residual)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= p.scale;
  if (!first) {
    float sum[N];
    load_values<ROW>(p.out, z, m, n, count, sum);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += sum[i];
  }
  if (last && p.bias) {
    if constexpr (ROW) {
      float b[N];
      load_values<true>(Plane{const_cast<void *>(p.bias), 0, 0, p.bias_type}, 0, 0, n, count, b);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += b[i];
    } else if (count > 0) {
      float b = 0.f;
      by_type(p.bias_type, [&](auto *type) {
        b = to_float(static_cast<const std::remove_pointer_t<decltype(type)> *>(p.bias)[n]);
      });
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += b;
    }
  }
  if (last && p.pre.p) store_values<ROW>(p.pre, z, m, n, count, x);
  if (last) activate(x, p.act);
  if (p.residual.p && (p.fold ? first : last)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += p.residual_scale * residual[i];
  }
  if (p.symmetric) {
    // This side of the diagonal, and its mirror image.
    by_type(p.out.type, [&](auto *type) {
      using T = std::remove_pointer_t<decltype(type)>;
      T *out = static_cast<T *>(p.out.p) + z * p.out.batch;
      if constexpr (ROW) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i < count && n + i <= m) from_float(out[m * p.out.stride + n + i], x[i]);
          if (i < count && n + i < m) from_float(out[(n + i) * p.out.stride + m], x[i]);
        }
      } else {
        T *dst = out + m * p.out.stride + n;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i < count && n <= m + i) from_float(*dst, x[i]);
          dst += p.out.stride;
        }
        dst = out + n * p.out.stride + m;
        if (sizeof(T) == 2 && count == N && n < m) {  // rows of 8 values on 16 bytes, as the operands'
          alignas(16) T v[N];
#pragma unroll
          for (int i = 0; i < N; ++i) from_float(v[i], x[i]);
#pragma unroll
          for (int i = 0; i < N; i += 8)
            *reinterpret_cast<uint4 *>(dst + i) = *reinterpret_cast<const uint4 *>(v + i);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i < count && n < m + i) from_float(dst[i], x[i]);
        }
      }
    });
  } else {
    store_values<ROW>(p.out, z, m, n, count, x);
  }
}

// A warp's part of an accumulator: 32 lanes (columns n, n + 1, .. of out), `chunks` times 16 of
// its rows from m0 on.  `release` runs once the last column is in registers, before its stores.
template <typename F>
__device__ __forceinline__ void drain(const ProductDev &p, uint32_t taddr, int chunks, int z, int m0, int n,
                                      bool first, bool last, F release) {
  const int rows = n < p.N ? min(chunks * 16, p.M - m0) : 0;
  const bool residual = p.residual.p && (p.fold ? first : last);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const int count = min(16, rows - c * 16);
    float r[16];
    if (residual) load_values<false>(p.residual, z, m0 + c * 16, n, count, r);
    uint32_t v[16];
    __syncwarp();  // together again after the stores, as tcgen05.ld wants the warp
    tmem_ld16(taddr + c * 16, v);
    if (c == chunks - 1) release();
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
    finish<false>(p, z, m0 + c * 16, n, count, first, last, x, r);
  }
}

// ---- the kernels ------------------------------------------------------------------------

// Barriers: full lives in the leader (the pair's even CTA; otherwise the CTA itself), with one
// arrival that expects both CTAs' bytes; empty, acc_full and mma_done exist in both and take the
// leader's multicast commits; acc_empty lives in the leader and takes an arrival from every
// epilogue warp of the pair.
template <bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(PAIR ? kPairThreads : kThreads, SPLIT ? 2 : 1)
    product_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ ProductDev p) {
  static_assert(!(PAIR && SPLIT));
  constexpr uint32_t kBudget = PAIR ? kPairStageBudget : SPLIT ? kSplitStageBudget : kStageBudget;
  constexpr uint32_t kCols = SPLIT ? kSplitTmemCols : kTmemCols;
  constexpr int kAccCols = PAIR ? kPairQMax : kQMax;
  constexpr int kTileP = PAIR ? 2 * kP : kP;
  constexpr int kParts = PAIR ? kPairParts : 1;
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + kBudget);
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.stages, qt = p.q_tile;
  const uint32_t stage_bytes = kPBytes + (uint32_t)p.q_rows * 128;
  const uint32_t rank = PAIR || SPLIT ? cluster_rank() : 0;
  // This CTA's blocks of K (from kb_first on) and its tiles.
  const int kb_first = SPLIT ? (int)((int64_t)p.kblocks * rank / p.splits) : 0;
  const int kblocks = SPLIT ? (int)((int64_t)p.kblocks * (rank + 1) / p.splits) - kb_first : p.kblocks;
  const int share = PAIR ? 2 : SPLIT ? p.splits : 1;  // CTAs a tile
  const int first_tile = blockIdx.x / share, tile_step = gridDim.x / share;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full + a, 1);
      mbar_init(acc_empty + a, (PAIR ? 2 : 1) * 4 * kParts);
    }
    mbar_init(mma_done, 1);
    if (p.withhold) mbar_expect_tx(full, 16);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers are initialised before either uses the other's
  else
    __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- TMA producer
      const uint32_t full_at = PAIR ? map_to_rank(smem_u32(full), 0) : smem_u32(full);
      uint32_t it = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
        Tile t = tile_at<kTileP>(p, tile);
        if constexpr (PAIR) t.p0 += rank * kP, t.q0 += rank * (qt / 2);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          if (!(ok = wait_phase(empty + s, ph ^ 1, abort_flag, p.wait_limit_ns, p.status))) break;
          const uint32_t st = smem_u32(sm) + s * stage_bytes, bar = full_at + 8u * s;
          if (rank == 0 || !PAIR) mbar_arrive_expect_tx(full + s, (PAIR ? 2 : 1) * stage_bytes);
          const int k = (kb_first + kb) * kBK;
          load_operand<PAIR>(st, &map_p, p.p_t, t.p0, kP, k, t.z, bar);
          load_operand<PAIR>(st + kPBytes, &map_q, p.q_t, t.q0, p.q_rows, k, t.z, bar);
          if (++s == stages) s = 0, ph ^= 1;
        }
      }
      // Loads issued into shared memory land before the block can exit (a pair's leader counts
      // both CTAs' bytes).
      if (rank == 0 || !PAIR)
        for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j)
          drain_phase(full + j % stages, (j / stages) & 1, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    if (rank == 0 || !PAIR) {
      // ---------------------------------------------------------- MMA issuer
      // The warp runs the loop together, so that what the instructions take is computed once in
      // its uniform registers; one lane issues.
      uint32_t unit = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const bool one = elect_one();
      const uint32_t p_step = desc_step(p.p_t), q_step = desc_step(p.q_t);
      for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
        for (int kb0 = 0; ok && kb0 < kblocks; kb0 += p.seg_blocks, ++unit) {
          const int kb1 = min(kb0 + p.seg_blocks, kblocks);
          const uint32_t acc = SPLIT ? 0 : unit & 1, use = unit >> 1;
          if (!(ok = warp_wait(acc_empty + acc, (use & 1) ^ 1, abort_flag, p))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t d = tmem + acc * kAccCols;
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = warp_wait(full + s, ph, abort_flag, p))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t st = smem_u32(sm) + s * stage_bytes;
            const uint64_t pd = operand_desc(st, p.p_t), qd = operand_desc(st + kPBytes, p.q_t);
            if (one) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f16<PAIR>(d, pd + k * p_step, qd + k * q_step, p.idesc, kb != kb0 || k != 0 ? 1u : 0u);
              commit<PAIR>(empty + s);
            }
            __syncwarp();
            if (++s == stages) s = 0, ph ^= 1;
          }
          if (ok && one) commit<PAIR>(acc_full + acc);
          __syncwarp();
        }
      }
      if (one) commit<PAIR>(mma_done);
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const uint32_t acc_empty_at = PAIR ? map_to_rank(smem_u32(acc_empty), 0) : smem_u32(acc_empty);
    // This warp's 16-column chunks: a part of the tile's.
    const int c0 = qt / 16 * part / kParts, chunks = qt / 16 * (part + 1) / kParts - c0;
    const uint32_t quad_tmem = tmem + ((uint32_t)(quad * 32) << 16);
    uint32_t unit = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < p.tiles; tile += tile_step) {
      const Tile t = tile_at<kTileP>(p, tile);
      const int n = t.p0 + (PAIR ? rank * kP : 0) + quad * 32 + lane;
      for (int seg = 0; seg < p.segments; ++seg, ++unit) {
        const uint32_t acc = SPLIT ? 0 : unit & 1, use = unit >> 1;
        ok = warp_wait(acc_full + acc, use & 1, abort_flag, p);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (SPLIT) {
          // The partial tile into shared memory (the stages: every MMA has read them).
          float *mine = reinterpret_cast<float *>(sm) + quad * 32 + lane;
          for (int c = 0; c < qt; c += 16) {
            uint32_t v[16];
            tmem_ld16(quad_tmem + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) mine[(c + i) * kP] = __uint_as_float(v[i]);
          }
          break;
        }
        drain(p, quad_tmem + acc * kAccCols + c0 * 16, chunks, t.z, t.q0 + c0 * 16, n, seg == 0,
              seg == p.segments - 1, [&] {
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                  if constexpr (PAIR)
                    mbar_arrive_cluster(acc_empty_at + 8u * acc);
                  else
                    mbar_arrive(acc_empty + acc);
                }
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
    const Tile t = tile_at<kTileP>(p, first_tile);
    // A warp a column (128 outputs of one row of out), four outputs a lane.
    const int n = t.p0 + lane * 4;
    const int q_end = qt * (rank + 1) / p.splits;
    for (int q = qt * rank / p.splits + warp; q < q_end; q += kThreads / 32) {
      const int m = t.q0 + q, count = ok && m < p.M ? min(4, p.N - n) : 0;
      const uint32_t at = smem_u32(sm) + (q * kP + lane * 4) * 4;
      float residual[4];
      if (p.residual.p) load_values<true>(p.residual, t.z, m, n, count, residual);
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = r < p.splits ? load4_cluster(map_to_rank(at, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 1; r < 8; ++r)
        v[0].x += v[r].x, v[0].y += v[r].y, v[0].z += v[r].z, v[0].w += v[r].w;
      float x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      finish<true>(p, t.z, m, n, count, true, true, x, residual);
    }
    cluster_sync();  // no CTA leaves while another may still read its part
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1 && lane == 0) drain_phase(mma_done, 0, p.wait_limit_ns);  // the MMAs ran
  __syncwarp();
  if constexpr (PAIR) cluster_sync();  // no CTA leaves while the other may still signal it
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1) {
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                   : "memory");
  }
}

// An operand as a 3-D tiled map (its fast dimension, the other, matrices) with 128-byte swizzle
// and zero fill outside: boxes of 64 of K x box_rows, or with `t` of 64 rows x 64 of K.
bool make_map(CUtensorMap *map, const Operand &o, int64_t rows, int64_t K, int64_t count, uint32_t box_rows) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const int64_t inner = o.t ? rows : K, outer = o.t ? K : rows;
  // One row or one matrix has no stride, but the map takes one all the same.
  const int64_t stride = outer > 1 ? o.stride : (inner + 7) / 8 * 8;
  const int64_t batch = count > 1 ? o.batch : stride * outer;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)batch * 2};
  const cuuint32_t box[3] = {64, o.t ? 64 : box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(o.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceInfo {
  bool ready = false;
  int sms = 0, pairs = 0;  // pairs: CTA pairs that fit at once
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
    constexpr auto attribute = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(product_kernel<false, false>, attribute, (int)kSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(product_kernel<false, true>, attribute, (int)kSplitSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(product_kernel<true, false>, attribute, (int)kPairSmemBytes);
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
    if ((e = cudaOccupancyMaxActiveClusters(&d.pairs, product_kernel<true, false>, &cfg)) != cudaSuccess) return e;
    d.ready = true;
  }
  out = d;
  return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of one matrix, `width` (along b) by qt (along a).
int64_t tiles_of(const ProductParams &p, int width, int qt) {
  const int64_t tp = ceil_div(p.N, width), tq = ceil_div(p.M, qt);
  if (!p.symmetric) return tp * tq;
  int64_t n = 0;
  for (int64_t q = 0; q < tq; ++q) {
    const int64_t end = p.M < (q + 1) * qt ? p.M : (q + 1) * qt, wide = (end - 1) / width + 1;
    n += tp < wide ? tp : wide;
  }
  return n;
}

bool overlaps(const Plane &a, const Plane &b, int64_t M, int64_t N) {
  const auto bytes = [&](const Plane &x) {
    return ((M - 1) * x.stride + N) * (x.type == ENGRAM_DTYPE_F32 ? 4 : 2);
  };
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x && y && x < y + bytes(b) && y < x + bytes(a);
}

}  // namespace

cudaError_t launch_product(const ProductParams &p, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(info);
  if (e != cudaSuccess) return e;
  ProductDev d{};
  d.out = p.out;
  d.residual = p.residual;
  d.pre = p.pre;
  d.bias = p.bias;
  d.bias_type = p.bias_type;
  d.act = p.act;
  d.scale = p.scale;
  d.residual_scale = p.residual_scale;
  d.status = p.status;
  d.wait_limit_ns = wait_limit_ns();
  d.withhold = take_withheld_launch();
  d.M = (int32_t)p.M;
  d.N = (int32_t)p.N;
  d.p_t = p.b.t;
  d.q_t = p.a.t;
  d.symmetric = p.symmetric;
  d.many = p.count > 1;
  d.kblocks = (int32_t)ceil_div(p.K, kBK);
  // Segments only where the output has the bits to show them, and nothing of it is needed later.
  const bool in_place = p.count == 1 && overlaps(p.out, p.residual, p.M, p.N);
  d.segments = 1;
  d.seg_blocks = d.kblocks;
  if (p.out.type == ENGRAM_DTYPE_F32 && !(in_place && (p.act != ENGRAM_ACT_NONE || p.pre.p))) {
    d.seg_blocks = (int32_t)ceil_div(d.kblocks, ceil_div(d.kblocks, kSegmentBlocks));
    d.segments = (int32_t)ceil_div(d.kblocks, d.seg_blocks);
    d.fold = in_place && d.segments > 1;
  }
  const double kb = d.kblocks;
  const int q_single = (int)(p.M < kQMax ? ceil_div(p.M, 16) * 16 : kQMax);
  const int64_t single_tiles = p.count * tiles_of(p, kP, q_single);
  const double single_us = ceil_div(single_tiles, info.sms) * (1.3 + 0.23 * kb);
  double pair_us = HUGE_VAL;
  if (info.pairs > 0 && p.M > 128 && p.N > 128) {
    for (int qt = kPairQMax; qt >= 128; qt -= 16) {
      const int64_t waves = ceil_div(p.count * tiles_of(p, 2 * kP, qt), info.pairs);
      const double us = 1.5 + waves * fmax(4.6 * qt / kPairQMax, 2.1 + fmax(0.2, 0.0013 * qt) * kb);
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
  if (!pair) d.q_tile = q_single;
  const int q_staged = pair ? d.q_tile / 2 : d.q_tile;
  d.q_rows = d.q_t ? (q_staged + 63) / 64 * 64 : q_staged;
  const uint32_t budget = pair ? kPairStageBudget : split ? kSplitStageBudget : kStageBudget;
  d.stages = (int32_t)(budget / (kPBytes + d.q_rows * 128));
  if (d.stages > kMaxStages) d.stages = kMaxStages;
  if (split) {  // a CTA's part of K is one segment
    d.segments = 1;
    d.seg_blocks = d.kblocks;
    d.fold = false;
  }
  const int width = pair ? 2 * kP : kP;
  const int64_t matrix_tiles = tiles_of(p, width, d.q_tile), tiles = matrix_tiles * p.count;
  if (tiles > INT32_MAX / 16) return cudaErrorInvalidConfiguration;
  d.tiles_p = (int32_t)ceil_div(p.N, width);
  d.tiles_q = (int32_t)ceil_div(p.M, d.q_tile);
  d.matrix_tiles = (int32_t)matrix_tiles;
  d.tiles = (int32_t)tiles;
  // kind::f16: fp32 accumulator, the operands' type (0: f16, 1: bf16), which of them are MN-major.
  d.idesc = 1u << 4 | (p.f16 ? 0u : 1u << 7 | 1u << 10) | (uint32_t)d.p_t << 15 | (uint32_t)d.q_t << 16 |
            (uint32_t)(d.q_tile >> 3) << 17 | (uint32_t)(width >> 4) << 24;
  CUtensorMap map_p, map_q;
  if (!make_map(&map_p, p.b, p.N, p.K, p.count, kP) ||
      !make_map(&map_q, p.a, p.M, p.K, p.count, (uint32_t)q_staged))
    return cudaErrorInvalidValue;
  if (pair)
    return launch(product_kernel<true, false>, 2 * (tiles < info.pairs ? tiles : info.pairs), kPairThreads,
                  kPairSmemBytes, stream, 2, map_p, map_q, d);
  if (split)
    return launch(product_kernel<false, true>, tiles * d.splits, kThreads, kSplitSmemBytes, stream, d.splits,
                  map_p, map_q, d);
  return launch(product_kernel<false, false>, tiles < info.sms ? tiles : info.sms, kThreads, kSmemBytes, stream, 1,
                map_p, map_q, d);
}

}  // namespace engram

// product.cu -- out = act(scale * a b^T + bias) + residual for 16-bit operands, on the sm_103a
// tensor cores (tcgen05.mma kind::f16, fp32 accumulators in TMEM).
//
// Where out, pre and residual have rows that start (and out and pre rows that end) on 16-byte
// boundaries and there are more than 64 rows, out's rows are the instruction's M rows and lie in the
// lanes of TMEM: tensor copies move 32 x 32 values at a time through shared memory.  Elsewhere the
// roles are turned around: out's columns lie in the lanes, and a warp of the epilogue holds 32
// neighbouring outputs of one row, which it reads and stores as whole lines for any stride and size.
// Either operand may run along K in memory (K-major) or along its rows (MN-major: boxes of 64 rows x
// 64 of K, told to the instruction by its descriptors), so the gradient's products and those of the
// symmetric iteration need no transposed copies.
//
// Two persistent kernels walk tiles of out; P stands for the operand whose rows are the lanes, Q for
// the other:
//   pairs: CTA pairs (tcgen05.mma.cta_group::2), tiles of 256 (P) x up to 256 (Q) values -- each CTA
//     stages its 128 rows of P and half of the rows of Q;
//   single: one CTA, 128 x up to 128 tiles, for products too small to fill the pairs; where even
//     those leave SMs idle (a few rows of a: reading b is the work), 2 to 8 CTAs of a cluster share a
//     tile, each with a part of K, and add their parts through distributed shared memory in rank
//     order, two such CTAs an SM.
// 65,536 x 4096 x 6144 takes 1790 to 1930 us in pairs, 1.7 to 1.8 PFLOP/s as the power limit lets it;
// 37 x 4096 x 6144 14.1 us, K shared by 8: 50 MB, 7.5 us at the measured bandwidth, behind the launch,
// the first bytes and the joining.
// Warps: 0, 2 and 3 TMA producers (a ring of stages of 64 of K, 128-byte swizzle); 1 allocates TMEM,
// one thread (of the pair's even CTA) issues the MMAs into one of two accumulators; 4.. epilogue.
//
// The fp32 accumulator of the tensor cores does not round to nearest: its error grows with the
// number of additions (1e-9 of the result for each value of K, against 1e-6 of an fp32 sum of
// 8192).  So where out or pre is fp32, K is cut into segments of at most 768 that each start a new
// accumulator, and the epilogue adds them in registers, rounding to nearest (7e-7 of the result;
// segments of 512 would be 5e-7 and take 4 % longer, of 1024 1e-6).  CTAs that share K put their part
// of it into two accumulators, or where it is longer than two segments into three or four.  16-bit
// outputs take segments of 262,144, about 8e-4 of a sum of like signs, a fifth of their rounding: one
// accumulator of 2^25 values is 1e-2 off.
//
// An operand may be the sum of two matrices (a gradient of which bf16 holds a half each): K goes
// through one and then the other, in the same accumulators.
//
// A symmetric product (both operands one matrix) computes the tiles on one side of the diagonal
// and stores every unit of 32 x 32 values twice, the second time turned in shared memory.
//
// Every wait is bounded as in wkv_gemm.cu: one that gives up sets ENGRAM_FLAG_TIMEOUT and leaves
// the tiles not yet stored unwritten.
#include <math.h>

#include <mutex>

#include "launch.cuh"
#include "product_internal.cuh"
#include "tensor_pieces.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kP = 128;         // rows of the P operand a CTA stages
constexpr int kBK = 64;         // of K a stage: 128 bytes
constexpr int kQMax = 128;      // most rows of the Q operand a tile of one CTA
constexpr int kPairQMax = 256;  // and of a pair
constexpr int kApartQMax = 64;  // and of CTAs that share K and have more than two accumulators
// Epilogue warps: one of each quarter of the lanes for each part of a tile's columns.
constexpr int kParts = 4, kPairParts = 4;
constexpr int kThreads = 128 * (1 + kParts), kPairThreads = 128 * (1 + kPairParts);
constexpr int kSplitParts = 2, kSplitThreads = 128 * (1 + kSplitParts);
constexpr int kSegmentBlocks = 12, kHalfSegmentBlocks = 4096;
constexpr int kMaxStages = 12, kMaxAhead = 4, kProducers = 3;
constexpr uint32_t kPBytes = kP * kBK * 2;
constexpr uint32_t kBarBytes = 1024;
constexpr int kUnit = 32;   // columns a warp of the tiles' epilogue moves at a time
// Shared memory for stages and epilogue buffers.
constexpr uint32_t kBudget = 224 * 1024;
constexpr uint32_t kSplitBudget = 104 * 1024;
constexpr uint32_t kTmemCols = 512, kSplitTmemCols = 256;
constexpr size_t kSmemBytes = 1024 + kBarBytes + kBudget;
constexpr size_t kSplitSmemBytes = 1024 + kBarBytes + kSplitBudget;
static_assert(2 * (kSplitSmemBytes + 1024) <= 228 * 1024 && kSmemBytes <= 227 * 1024);
static_assert(kSplitBudget >= kProducers * 2 * kPBytes &&
              kBudget >= kProducers * 2 * kPBytes + 4 * kPairParts * 2 * 32 * kUnit * 4);
static_assert(kParts <= kPairParts && (2 * kMaxStages + 6 + 4 * kPairParts * kMaxAhead) * 8 + 8 <= kBarBytes);

struct PlaneDev {
  void *p;
  int64_t stride, batch;
  int32_t type;
  bool vec;  // rows start on 16-byte boundaries
};

struct ProductDev {
  PlaneDev out, residual, pre, bias;
  int32_t *status;
  int64_t wait_limit_ns;
  int32_t M, N;
  float scale, residual_scale;
  int32_t act;
  int32_t kblocks, q_tile, q_rows, stages;  // q_rows: rows of Q that a CTA stages
  // Blocks of K of one matrix.  Where an operand is the sum of two, K goes on from the first to the
  // second (p_next, q_next: 1), and begins anew in the other.
  int32_t pass_blocks, p_next, q_next;
  int32_t segments, seg_blocks;  // of a split product: the accumulators that a CTA's part of K goes into
  int32_t tiles_p, tiles_q, tiles, matrix_tiles;
  // tiles of a group of out's columns; how many columns of tiles it has, and the last one
  int32_t group_columns, group_tiles, last_columns;
  FastDiv by_matrix, by_group, by_columns, by_last;
  uint32_t idesc;
  // the tiles' epilogue: of each warp, buffers for units of the residual ahead (ahead of them,
  // ahead_bytes each) and for units on their way out (slots of them, slot_bytes each)
  int32_t ahead, slots;
  uint32_t ahead_bytes, slot_bytes;
  // which CTAs (or pairs) take which tiles: see Walk
  int32_t shift, extra;
  bool p_t, q_t, many;
  const float *diag_in;  // as in ProductParams
  float *diag_out;
  int64_t diag_batch;
  float diag_by, diag_scale;
  bool diag_rows, diag_columns;
  bool rows;      // rows of out in the lanes; else its columns
  bool withhold;  // test hook: the first stage waits for bytes that never come
};

// One product, or two that share a launch.
struct Job {
  CUtensorMap p, q, out, pre, residual;
  ProductDev d;
};
struct Jobs {
  Job job[2];
  int32_t count, stages, splits;
  // warp_bytes: buffers of an epilogue warp, the larger of both jobs'.  A warp keeps its own from one
  // job to the next: nothing orders it against the others there, whose copies may be on their way.
  uint32_t stage_bytes, warp_bytes;
};

// Shared-memory descriptor of an operand tile, 128-byte swizzle.  K-major: rows of 64 of K,
// 8-row groups 1024 bytes apart.  MN-major: boxes of 64 rows (128 bytes) by 64 of K, 8192 bytes
// apart along the rows, groups of 8 along K 1024 bytes apart.  The halves: address and the stride
// between boxes; the stride between groups, descriptor version 1, SWIZZLE_128B (2).
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, bool t) {
  return ((addr >> 4) & 0x3FFF) | (uint32_t)(t ? 8192 >> 4 : 1) << 16;
}
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// What 16 of K add to it, in its units of 16 bytes.
__device__ __forceinline__ uint32_t desc_step(bool t) { return t ? 2048 >> 4 : 32 >> 4; }

template <bool PAIR>
__device__ __forceinline__ void umma_f16(uint32_t d, uint32_t p_low, uint32_t q_low, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(p_low), "r"(q_low), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(p_low), "r"(q_low), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
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

// The whole warp waits; the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                          const ProductDev &p) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p.wait_limit_ns, p.status));
}

struct Tile {
  int p0, q0, z;
};
// Tiles in groups of up to group_columns along out's columns, inside a group row by row: the resident CTAs
// read a few slices of a at a time, once, and a group of slices of b that stays in L2.  Of a
// symmetric product those that hold any output (m, n) with n <= m.
template <int WIDTH, bool SYMMETRIC>
__device__ __forceinline__ Tile tile_at(const ProductDev &p, int tile) {
  Tile r{0, 0, 0};
  uint32_t t = tile;
  if (p.many) {
    r.z = fast_div(t, p.by_matrix);
    t -= r.z * (uint32_t)p.matrix_tiles;
  }
  uint32_t tp, tq;
  if constexpr (SYMMETRIC) {
    for (tp = 0;; ++tp) {
      const uint32_t wide = min(p.tiles_q, (min(p.M, (int)(tp + 1) * WIDTH) - 1) / p.q_tile + 1);
      if (t < wide) break;
      t -= wide;
    }
    tq = t;
  } else {
    const uint32_t g = fast_div(t, p.by_group), in = t - g * p.group_tiles, before = g * p.group_columns;
    const bool last = before + p.group_columns > (uint32_t)(p.rows ? p.tiles_q : p.tiles_p);
    const uint32_t row = fast_div(in, last ? p.by_last : p.by_columns);
    const uint32_t column = before + in - row * (last ? p.last_columns : p.group_columns);
    tp = p.rows ? row : column, tq = p.rows ? column : row;
  }
  r.p0 = (int)tp * WIDTH, r.q0 = (int)tq * p.q_tile;
  return r;
}

// The tiles of worker w of `workers` (CTAs or pairs).  One after the other in steps of `workers`;
// but of a second product the workers from `shift` on, which had a tile less of the first, take
// `extra` more each before that, and the others come last.
struct Walk {
  int tile, left, step, rest, lights;

  __device__ __forceinline__ Walk(const ProductDev &p, int w, int workers) {
    lights = workers - p.shift;
    step = workers;
    const int turn = w >= p.shift ? w - p.shift : w + lights;
    rest = p.extra * lights + turn;
    left = w >= p.shift ? p.extra : 0;
    tile = left ? turn : rest;
  }
  __device__ __forceinline__ void next() {
    if (left > 1)
      tile += lights;
    else if (left == 1)
      tile = rest;
    else
      tile += step;
    if (left) --left;
  }
};

// ---- epilogue ---------------------------------------------------------------------------

// How a kernel's epilogue moves its values.
//   tiles: the lanes of TMEM are rows of out.  A lane turns 32 values of its row into words that it
//     puts into shared memory, from where tensor copies take 32 x 32 values at a time to out (and
//     pre); the residual comes in the same way, asked for ahead.  Where their rows lie on 16-byte
//     boundaries.
//   singles: the lanes of TMEM are columns of out.  A warp moves 32 neighbouring values of a row at a
//     time: any strides, few rows, sums in segments.
// A symmetric product takes the first, with a second store of each unit below the diagonal.

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

__device__ __forceinline__ uint8_t *element(const PlaneDev &s, int64_t z, int64_t m, int64_t n) {
  return static_cast<uint8_t *>(s.p) + ((z * s.batch + m * s.stride + n) << (s.type == ENGRAM_DTYPE_F32 ? 2 : 1));
}
__device__ __forceinline__ float load_one(const PlaneDev &s, int64_t z, int64_t m, int64_t n) {
  const uint8_t *at = element(s, z, m, n);
  if (s.type == ENGRAM_DTYPE_F32) return *reinterpret_cast<const float *>(at);
  const uint16_t v = *reinterpret_cast<const uint16_t *>(at);
  return s.type == ENGRAM_DTYPE_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ void store_one(const PlaneDev &d, int64_t z, int64_t m, int64_t n, float v) {
  by_type(d.type, [&](auto *type) { from_float(*reinterpret_cast<decltype(type)>(element(d, z, m, n)), v); });
}

__device__ __forceinline__ void decode2(uint32_t w, int type, float &lo, float &hi) {
  if (type == ENGRAM_DTYPE_BF16) {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  } else {
    lo = __half2float(__ushort_as_half((uint16_t)w)), hi = __half2float(__ushort_as_half((uint16_t)(w >> 16)));
  }
}
// Two neighbouring 16-bit values, rounded to nearest even.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
  if (type == ENGRAM_DTYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <int N>
__device__ __forceinline__ void activate(float (&x)[N], int act) {
  if (act == ENGRAM_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = activated(x[i], ENGRAM_ACT_RELU);
  } else if (act == ENGRAM_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = activated(x[i], ENGRAM_ACT_SILU);
  } else if (act == ENGRAM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = activated(x[i], ENGRAM_ACT_GELU);
  }
}

// ---- tiles

// Where 16-byte piece j of row r of a unit lies: rows of 64 or 128 bytes (F32), swizzled as the
// tensor copies do.
template <bool F32>
__device__ __forceinline__ uint32_t piece(uint32_t unit, int r, int j) {
  return F32 ? unit + r * 128 + ((j ^ (r & 7)) << 4) : unit + r * 64 + ((j ^ (r >> 1 & 3)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// A lane's 32 values of row r of a unit, rounded to `type`.
__device__ __forceinline__ void put_row(uint32_t unit, int r, int type, const float (&x)[kUnit]) {
  if (type == ENGRAM_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared(piece<true>(unit, r, j), __float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared(piece<false>(unit, r, j), pack2(x[8 * j], x[8 * j + 1], type), pack2(x[8 * j + 2], x[8 * j + 3], type),
                pack2(x[8 * j + 4], x[8 * j + 5], type), pack2(x[8 * j + 6], x[8 * j + 7], type));
  }
}
// The same as column r of a unit, rounded to fp16: in every row a lane's value lies beside its
// neighbours'.
__device__ __forceinline__ void put_column(uint32_t unit, int r, const float (&x)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i)
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(piece<false>(unit, i, r >> 3) + (r & 7) * 2),
                 "h"(__half_as_ushort(__float2half_rn(x[i])))
                 : "memory");
}
// x += by(m, n) * the row's fp16 values: base and, where there is d, `column` times a column's value of d.
__device__ __forceinline__ void add_row_by(uint32_t unit, int r, float base, float column, const float *d,
                                           float (&x)[kUnit]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = ld_shared(piece<false>(unit, r, j));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float by[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) by[i] = base;
    if (d) {
      const float4 d0 = reinterpret_cast<const float4 *>(d)[2 * j], d1 = reinterpret_cast<const float4 *>(d)[2 * j + 1];
      const float all[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) by[i] = fmaf(column, all[i], base);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      decode2(w[i], kTypeF16, lo, hi);
      x[8 * j + 2 * i] = fmaf(by[2 * i], lo, x[8 * j + 2 * i]);
      x[8 * j + 2 * i + 1] = fmaf(by[2 * i + 1], hi, x[8 * j + 2 * i + 1]);
    }
  }
}
// What diag_out receives of an element (m, m) and its value d of diag_in.
__device__ __forceinline__ float on_diagonal(const ProductDev &p, float x, float d) {
  return fmaf(fmaf(p.diag_by, d, p.residual_scale), d, x * p.diag_scale);
}
// x += by * the row's values.
__device__ __forceinline__ void add_row(uint32_t unit, int r, int type, float by, float (&x)[kUnit]) {
  if (type == ENGRAM_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 v = ld_shared(piece<true>(unit, r, j));
      x[4 * j] = fmaf(by, __uint_as_float(v.x), x[4 * j]);
      x[4 * j + 1] = fmaf(by, __uint_as_float(v.y), x[4 * j + 1]);
      x[4 * j + 2] = fmaf(by, __uint_as_float(v.z), x[4 * j + 2]);
      x[4 * j + 3] = fmaf(by, __uint_as_float(v.w), x[4 * j + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 v = ld_shared(piece<false>(unit, r, j));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        decode2(w[i], type, lo, hi);
        x[8 * j + 2 * i] = fmaf(by, lo, x[8 * j + 2 * i]);
        x[8 * j + 2 * i + 1] = fmaf(by, hi, x[8 * j + 2 * i + 1]);
      }
    }
  }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// What a warp moves of its CTA's tiles, unit by unit (32 rows x 32 columns): units [first, end) of
// each tile, `row0` rows into it.  Units that lie outside out are passed over, of a symmetric product
// those above the diagonal.
template <int WIDTH, bool SYMMETRIC>
struct Units {
  Walk walk;
  int unit, first, end, row0;
  Tile at;

  __device__ __forceinline__ Units(const ProductDev &p, const Walk &w, int first_, int end_, int row0_)
      : walk(w), unit(first_), first(first_), end(end_), row0(row0_) {
    if (walk.tile < p.tiles) at = tile_at<WIDTH, SYMMETRIC>(p, walk.tile);
  }
  __device__ __forceinline__ bool done(const ProductDev &p) const { return walk.tile >= p.tiles; }
  __device__ __forceinline__ int n() const { return at.q0 + unit * kUnit; }
  __device__ __forceinline__ int m() const { return at.p0 + row0; }
  __device__ __forceinline__ bool inside(const ProductDev &p) const {
    return n() < p.N && m() < p.M && (!SYMMETRIC || n() <= m());
  }
  __device__ __forceinline__ void next(const ProductDev &p) {
    if (++unit < end) return;
    unit = first;
    walk.next();
    if (walk.tile < p.tiles) at = tile_at<WIDTH, SYMMETRIC>(p, walk.tile);
  }
};

// An epilogue warp's place in what it shares with the rest of its CTA.
struct Shared {
  uint32_t buffers;           // its shared memory
  uint64_t *arrived;          // its barriers, one a residual buffer
  uint64_t *acc_full;
  uint32_t tmem;              // its quarter of the lanes
  int lane, row0;             // row0: its first lane, of the tile
  volatile int *abort_flag;
  uint32_t unit, phases;      // accumulators drained so far; the parities of `arrived`
};

// How a warp moves units: its buffers for what comes in (`ahead` of them) and goes out.
template <bool SYMMETRIC, bool NEWTON>
struct Mover {
  const Job &job;
  const ProductDev &p;
  Shared &w;
  int asked = 0, used = 0, slot = 0, waiting = 0;

  __device__ __forceinline__ Mover(const Job &j, Shared &shared) : job(j), p(j.d), w(shared) {}

  // Asks for the residual of a unit.
  __device__ __forceinline__ void ask(int n, int m, int z) {
    if (w.lane == 0) {
      if (p.slots == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      mbar_arrive_expect_tx(w.arrived + asked, p.ahead_bytes);
      tma_load_3d<false>(w.buffers + asked * p.ahead_bytes, &job.residual, n, m, z, smem_u32(w.arrived + asked));
    }
    asked = asked + 1 == p.ahead ? 0 : asked + 1;
    ++waiting;
  }

  // A free buffer: of the stores before, all but slots - 1 have been read.
  __device__ __forceinline__ uint32_t free_slot() {
    if (w.lane == 0) {
      if (p.slots == 1)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      else
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    }
    __syncwarp();
    const uint32_t at = w.buffers + p.ahead * p.ahead_bytes + slot * p.slot_bytes;
    slot = slot + 1 == p.slots ? 0 : slot + 1;
    return at;
  }
  __device__ __forceinline__ void send(const CUtensorMap *map, uint32_t from, int n, int m, int z) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (w.lane == 0) tma_store_3d(map, from, n, m, z);
  }

  __device__ __forceinline__ void add_bias(int n, float (&x)[kUnit]) {
    if (n + kUnit <= p.N && p.bias.vec) {  // the same 32 values in every lane
      if (p.bias.type == ENGRAM_DTYPE_F32) {
        const float4 *at = reinterpret_cast<const float4 *>(static_cast<const float *>(p.bias.p) + n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 b = __ldg(at + j);
          x[4 * j] += b.x, x[4 * j + 1] += b.y, x[4 * j + 2] += b.z, x[4 * j + 3] += b.w;
        }
      } else {
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.bias.p) + n);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 b = __ldg(at + j);
          const uint32_t words[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[8 * j + 2 * i] += __uint_as_float(words[i] << 16);
            x[8 * j + 2 * i + 1] += __uint_as_float(words[i] & 0xffff0000u);
          }
        }
      }
    } else {
      // A lane a value; past the edge nothing is kept.
      const float mine = n + w.lane < p.N ? load_one(p.bias, 0, 0, n + w.lane) : 0.f;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) x[i] += __shfl_sync(0xffffffffu, mine, i);
    }
  }

  // Sums of products of the unit at (m, n) become outputs; false if its residual did not arrive.
  __device__ __forceinline__ bool finish(int n, int m, int z, float (&x)[kUnit]) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) x[i] *= p.scale;
    if (p.bias.p) add_bias(n, x);
    if (p.pre.p) {
      const uint32_t at = free_slot();
      put_row(at, w.lane, p.pre.type, x);
      send(&job.pre, at, n, m, z);
    }
    activate(x, p.act);
    [[maybe_unused]] float d = 0.f;  // of the lane's row
    if (NEWTON && p.diag_rows) d = p.diag_in[z * p.diag_batch + m + w.lane];
    uint32_t at = 0;
    if (p.ahead) {
      if (!warp_wait(w.arrived + used, (w.phases >> used) & 1, w.abort_flag, p)) return false;
      w.phases ^= 1u << used;
      at = w.buffers + used * p.ahead_bytes;
      if constexpr (NEWTON)
        add_row_by(at, w.lane, fmaf(p.diag_by, d, p.residual_scale), p.diag_by,
                   p.diag_columns ? p.diag_in + z * p.diag_batch + n : nullptr, x);
      else
        add_row(at, w.lane, p.residual.type, p.residual_scale, x);
      used = used + 1 == p.ahead ? 0 : used + 1;
      --waiting;
      __syncwarp();
    }
    if (NEWTON && p.diag_out && n == m) {  // units lie on multiples of 32
      float own = 0.f;
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (i == w.lane) own = x[i], x[i] = 0.f;
      if (m + w.lane < p.M) p.diag_out[z * p.diag_batch + m + w.lane] = on_diagonal(p, own, d);
    }
    if (p.slots) at = free_slot();  // else out goes where the residual came
    put_row(at, w.lane, p.out.type, x);
    send(&job.out, at, n, m, z);
    if (SYMMETRIC && n < m) {  // and its mirror image
      const uint32_t turned = free_slot();
      put_column(turned, w.lane, x);
      send(&job.out, turned, m, n, z);
    }
    return true;
  }

  // What is on its way into shared memory has arrived, and what leaves it has been read, before
  // the buffers serve anything else and before the block exits.
  __device__ __forceinline__ void end() {
    if (w.lane == 0) {
      for (; waiting > 0; --waiting) {  // after a wait that gave up
        drain_phase(w.arrived + used, (w.phases >> used) & 1, p.wait_limit_ns);
        used = used + 1 == p.ahead ? 0 : used + 1;
      }
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
  }
};

// A warp's share of the epilogue of all of its CTA's tiles: units [first, end) of each.
template <bool PAIR, bool SYMMETRIC, bool NEWTON, typename F>
__device__ __forceinline__ bool move_tiles(const Job &job, const Walk &walk, Shared &w, int first, int end, F release) {
  constexpr int kWidth = PAIR ? 2 * kP : kP, kAccCols = PAIR ? kPairQMax : kQMax;
  const ProductDev &p = job.d;
  if (first == end) {  // a narrow tile has nothing for this part
    for (Walk k = walk; k.tile < p.tiles; k.next()) {
      const uint32_t acc = w.unit & 1;
      if (!warp_wait(w.acc_full + acc, (w.unit >> 1) & 1, w.abort_flag, p)) return false;
      release(acc);
      ++w.unit;
    }
    return true;
  }
  Mover<SYMMETRIC, NEWTON> mover(job, w);
  Units<kWidth, SYMMETRIC> ahead(p, walk, first, end, w.row0), now = ahead;
  // The residual of the next unit that has not been asked for.
  const auto ask = [&] {
    while (!ahead.done(p) && !ahead.inside(p)) ahead.next(p);
    if (ahead.done(p)) return;
    mover.ask(ahead.n(), ahead.m(), ahead.at.z);
    ahead.next(p);
  };
  for (int i = 0; i < p.ahead; ++i) ask();
  bool ok = true;
  for (; !now.done(p); now.next(p)) {
    const uint32_t acc = w.unit & 1;
    if (now.unit == first) {
      if (!(ok = warp_wait(w.acc_full + acc, (w.unit >> 1) & 1, w.abort_flag, p))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    uint32_t v[kUnit];
    __syncwarp();
    tmem_ld32(w.tmem + acc * kAccCols + now.unit * kUnit, v);
    if (now.unit == end - 1) {
      release(acc);
      ++w.unit;
    }
    if (!now.inside(p)) continue;
    float x[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) x[i] = __uint_as_float(v[i]);
    if (!(ok = mover.finish(now.n(), now.m(), now.at.z, x))) break;
    if (p.ahead) ask();
  }
  mover.end();
  return ok;
}

// Adds a tile's segments: `chunks` times 16 columns of the accumulators from `column` on.
template <int KACC, int COLUMNS, typename F>
__device__ __forceinline__ bool add_segments(const ProductDev &p, Shared &w, int column, int chunks,
                                             float (&sums)[COLUMNS], F release) {
#pragma unroll
  for (int i = 0; i < COLUMNS; ++i) sums[i] = 0.f;
#pragma unroll 1
  for (int seg = 0; seg < p.segments; ++seg, ++w.unit) {
    const uint32_t acc = w.unit & 1;
    if (!warp_wait(w.acc_full + acc, (w.unit >> 1) & 1, w.abort_flag, p)) return false;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
    for (int c = 0; c < COLUMNS / 16; ++c)
      if (c < chunks) {
        uint32_t v[16];
        tmem_ld16(w.tmem + acc * KACC + column + c * 16, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[c * 16 + i] += __uint_as_float(v[i]);
      }
    release(acc);
  }
  return true;
}

// move_tiles for products in segments, whose sums stay in registers.
template <bool PAIR, bool NEWTON, typename F>
__device__ __forceinline__ bool move_tiles_of_segments(const Job &job, Walk walk, Shared &w, int first, int end,
                                                       F release) {
  constexpr int kWidth = PAIR ? 2 * kP : kP, kAccCols = PAIR ? kPairQMax : kQMax;
  constexpr int kMost = kAccCols / kUnit / (PAIR ? kPairParts : kParts);  // units a warp
  const ProductDev &p = job.d;
  Mover<false, NEWTON> mover(job, w);
  bool ok = true;
  for (; ok && walk.tile < p.tiles; walk.next()) {
    const Tile t = tile_at<kWidth, false>(p, walk.tile);
    const int m = t.p0 + w.row0, n0 = t.q0 + first * kUnit;
    const int units = m < p.M ? min(end - first, (p.N - n0 + kUnit - 1) / kUnit) : 0;  // inside
    if (p.ahead && units > 0) mover.ask(n0, m, t.z);
    float sums[kMost * kUnit];
    ok = add_segments<kAccCols>(p, w, first * kUnit, 2 * (end - first), sums, release);
#pragma unroll 1
    for (int u = 0; ok && u < units; ++u) {
      float x[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) x[i] = sums[i];
#pragma unroll
      for (int i = kUnit; i < kMost * kUnit; ++i) sums[i - kUnit] = sums[i];  // the next unit's
      ok = mover.finish(n0 + u * kUnit, m, t.z, x);
      if (p.ahead && u + 1 < units) mover.ask(n0 + (u + 1) * kUnit, m, t.z);
    }
  }
  mover.end();
  return ok;
}

// ---- singles

// 16 values of one column of out, from row m on, of which `count` are there.
__device__ __forceinline__ void load_column(const PlaneDev &s, int z, int m, int n, int count, float (&x)[16]) {
  by_type(s.type, [&](auto *type) {
    auto *src = reinterpret_cast<decltype(type)>(element(s, z, m, n));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i < count ? to_float(*src) : 0.f;
      src += s.stride;
    }
  });
}
__device__ __forceinline__ void store_column(const PlaneDev &d, int z, int m, int n, int count,
                                             const float (&x)[16]) {
  by_type(d.type, [&](auto *type) {
    auto *dst = reinterpret_cast<decltype(type)>(element(d, z, m, n));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < count) from_float(*dst, x[i]);
      dst += d.stride;
    }
  });
}
// How many times the residual's 16 values count: NEWTON by diagonals, `own` the column's.
template <bool NEWTON>
struct Counts {
  float by[NEWTON ? 16 : 1], own;
  __device__ __forceinline__ Counts(const ProductDev &p, int z, int m, int n, int count) {
    if constexpr (NEWTON) {
      const float *d = p.diag_in + z * p.diag_batch;
      own = p.diag_columns && count > 0 ? d[n] : 0.f;
      const float base = fmaf(p.diag_by, own, p.residual_scale);
#pragma unroll
      for (int i = 0; i < 16; ++i) by[i] = base;
      if (p.diag_rows && count > 0) {  // m is a multiple of 16, and d's length one of 64
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4 *>(d + m + 4 * i);
          by[4 * i] = fmaf(p.diag_by, v.x, base), by[4 * i + 1] = fmaf(p.diag_by, v.y, base);
          by[4 * i + 2] = fmaf(p.diag_by, v.z, base), by[4 * i + 3] = fmaf(p.diag_by, v.w, base);
        }
      }
    }
  }
};

// Sums of products (m .., n) become outputs; y: the residual.
template <bool NEWTON>
__device__ __forceinline__ void finish_column(const ProductDev &p, int z, int m, int n, int count, float bias,
                                              float (&x)[16], const float (&y)[16], const Counts<NEWTON> &counts) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = fmaf(p.scale, x[i], bias);
  if (p.pre.p) store_column(p.pre, z, m, n, count, x);
  activate(x, p.act);
  if (p.residual.p) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf(NEWTON ? counts.by[NEWTON ? i : 0] : p.residual_scale, y[i], x[i]);
  }
  if constexpr (NEWTON) {
    if (p.diag_out && n >= m && n < m + count) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (m + i == n) {
          p.diag_out[z * p.diag_batch + n] = on_diagonal(p, x[i], counts.own);
          x[i] = 0.f;
        }
    }
  }
  store_column(p.out, z, m, n, count, x);
}

// A warp's share of a tile: column n of each lane, `chunks` times 16 rows from m0 on.  SEGMENTS: adds
// up the accumulators of a tile first.
template <int KACC, int MOST, bool SEGMENTS, bool NEWTON, typename F>
__device__ __forceinline__ bool drain_columns(const ProductDev &p, Shared &w, int z, int m0, int n, int column,
                                              int chunks, F release) {
  const bool there = n < p.N;
  const float bias = p.bias.p && there ? load_one(p.bias, 0, 0, n) : 0.f;
  if constexpr (SEGMENTS) {
    float sums[MOST * 16];
    if (!add_segments<KACC>(p, w, column, chunks, sums, release)) return false;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int m = m0 + c * 16, count = there ? min(16, p.M - m) : 0;
      float x[16], y[16];
      if (p.residual.p) load_column(p.residual, z, m, n, count, y);
      const Counts<NEWTON> counts(p, z, m, n, count);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = sums[i];
#pragma unroll
      for (int i = 16; i < MOST * 16; ++i) sums[i - 16] = sums[i];
      finish_column<NEWTON>(p, z, m, n, count, bias, x, y, counts);
    }
  } else {
    const uint32_t acc = w.unit & 1;
    if (!warp_wait(w.acc_full + acc, (w.unit >> 1) & 1, w.abort_flag, p)) return false;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int m = m0 + c * 16, count = there ? min(16, p.M - m) : 0;
      float x[16], y[16];
      if (p.residual.p) load_column(p.residual, z, m, n, count, y);
      const Counts<NEWTON> counts(p, z, m, n, count);
      uint32_t v[16];
      __syncwarp();  // together again after the stores, as tcgen05.ld wants the warp
      tmem_ld16(w.tmem + acc * KACC + column + c * 16, v);
      if (c == chunks - 1) release(acc);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
      finish_column<NEWTON>(p, z, m, n, count, bias, x, y, counts);
    }
    if (chunks == 0) release(acc);  // a narrow tile has nothing for this part
    ++w.unit;
  }
  return true;
}

__device__ __noinline__ float activated_apart(float x, int act) { return activated(x, act); }

// One sum of products of a tile that several CTAs share becomes an output.
template <bool NEWTON>
__device__ __forceinline__ void finish_one(const ProductDev &p, int64_t z, int64_t m, int64_t n, float x, float bias,
                                           float residual) {
  if constexpr (NEWTON) {  // nothing but a residual comes to it
    const float *d = p.diag_in + z * p.diag_batch;
    const float own = p.diag_rows ? d[m] : 0.f;
    x = fmaf(fmaf(p.diag_by, own + (p.diag_columns ? d[n] : 0.f), p.residual_scale), residual, x);
    if (p.diag_out && m == n) {
      p.diag_out[z * p.diag_batch + m] = on_diagonal(p, x, own);
      x = 0.f;
    }
    store_one(p.out, z, m, n, x);
    return;
  }
  x += bias;
  if (p.pre.p) store_one(p.pre, z, m, n, x);
  if (p.act != ENGRAM_ACT_NONE) x = activated_apart(x, p.act);
  store_one(p.out, z, m, n, x + residual);
}

// ---- the kernels ------------------------------------------------------------------------

// Barriers: full lives in the leader (the pair's even CTA; otherwise the CTA itself), with one
// arrival that expects both CTAs' bytes; empty, acc_full and mma_done exist in both and take the
// leader's multicast commits; acc_empty lives in the leader and takes an arrival from every
// epilogue warp of the pair.
// Of the products that a kernel is for: sums of segments of K; the iteration's (ProductParams::newton),
// symmetric ones among them.
enum Variant { kPlain, kSegments, kSymmetric, kNewton, kNewtonSegments, kVariants };

template <bool PAIR, bool SPLIT, int VARIANT>
__global__ void __launch_bounds__(PAIR ? kPairThreads : SPLIT ? kSplitThreads : kThreads, SPLIT ? 2 : 1)
    product_kernel(const __grid_constant__ Jobs jobs) {
  constexpr bool SYMMETRIC = VARIANT == kSymmetric, SEGMENTS = VARIANT == kSegments || VARIANT == kNewtonSegments;
  constexpr bool NEWTON = VARIANT >= kSymmetric;
  static_assert(!(PAIR && SPLIT) && !(SPLIT && (SYMMETRIC || VARIANT == kNewtonSegments)));
  constexpr bool kApart = SPLIT && SEGMENTS;  // more accumulators than two for a part of K
  constexpr uint32_t kCols = SPLIT ? kSplitTmemCols : kTmemCols;
  [[maybe_unused]] constexpr int kAccCols = PAIR ? kPairQMax : SPLIT && SEGMENTS ? kApartQMax : kQMax;
  constexpr int kTileP = PAIR ? 2 * kP : kP;
  constexpr int kPartsHere = PAIR ? kPairParts : SPLIT ? kSplitParts : kParts;
  constexpr int kThreadsHere = 128 * (1 + kPartsHere);
  extern __shared__ uint8_t sm_raw[];
  // Barriers, stages, the epilogue's buffers.
  uint8_t *base = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023), *sm = base + kBarBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(base);
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint64_t *arrived = mma_done + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(arrived + 4 * kPairParts * kMaxAhead);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = jobs.stages, splits = jobs.splits;
  const uint32_t stage_bytes = jobs.stage_bytes;
  const uint32_t rank = PAIR || SPLIT ? cluster_rank() : 0;
  const int share = PAIR ? 2 : SPLIT ? splits : 1;  // CTAs a tile
  const int worker = blockIdx.x / share, workers = gridDim.x / share;
  // Two products have their code each: what they read of their parameters stays constant operands.
  constexpr bool kTwo = !SPLIT && !NEWTON;
  // This CTA's blocks of K of a product.
  const auto first_block = [&](const ProductDev &p) {
    return SPLIT ? (int)((int64_t)p.kblocks * rank / splits) : 0;
  };
  const auto blocks = [&](const ProductDev &p) {
    return SPLIT ? (int)((int64_t)p.kblocks * (rank + 1) / splits) - first_block(p) : p.kblocks;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full + a, 1);
      mbar_init(acc_empty + a, (PAIR ? 2 : 1) * 4 * kPartsHere);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < 4 * kPartsHere * kMaxAhead; ++i) mbar_init(arrived + i, 1);
    if (jobs.job[0].d.withhold) mbar_expect_tx(full, 16);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >= 96 && threadIdx.x < 96 + jobs.count) {
    const Job &job = jobs.job[threadIdx.x - 96];
    const CUtensorMap *maps[4] = {&job.p, &job.q, job.d.rows ? &job.out : nullptr,
                                  job.d.rows && job.d.ahead ? &job.residual : nullptr};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (maps[i]) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
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

  if (warp < 4 && warp != 1) {
    if (lane == 0) {
      // ------------------------------------------------------- TMA producers
      // kProducers threads, a stage each in turn: one alone takes 180 ns a stage (waiting, expecting
      // its bytes, issuing its copies), whatever the stage holds.  The ring has at least as many
      // stages: a thread that waits for a stage to be free has seen the one kProducers before it
      // freed, so the phase two before the one it waits for, of the same parity, is over.
      const uint32_t full_at = PAIR ? map_to_rank(smem_u32(full), 0) : smem_u32(full);
      const int64_t limit = jobs.job[0].d.wait_limit_ns;
      uint32_t it = 0;
      int s = 0, turn = warp == 0 ? 0 : warp - 1;  // stages to go to the next one of this thread
      uint32_t ph = 0;
      bool ok = true;
      const auto produce = [&](const Job &job) {
        const ProductDev &p = job.d;
        const int kb_first = first_block(p), kblocks = blocks(p), q_rows = p.q_rows;
        const uint32_t bytes = (PAIR ? 2 : 1) * (kPBytes + (uint32_t)q_rows * 128);
        const bool p_t = p.p_t, q_t = p.q_t;
        const int pass = kb_first >= p.pass_blocks, k_end = p.pass_blocks * kBK;
        for (Walk walk(p, worker, workers); ok && walk.tile < p.tiles; walk.next()) {
          Tile at = tile_at<kTileP, SYMMETRIC>(p, walk.tile);
          if constexpr (PAIR) at.p0 += rank * kP, at.q0 += rank * (p.q_tile / 2);
          int k = (kb_first - pass * p.pass_blocks) * kBK;
          int pz = at.z + pass * p.p_next, qz = at.z + pass * p.q_next;
          for (int kb = 0; kb < kblocks; ++kb, ++it, k += kBK) {
            if (k == k_end) k = 0, pz += p.p_next, qz += p.q_next;
            if (turn == 0) {
              if (!(ok = wait_phase(empty + s, ph ^ 1, abort_flag, limit, p.status))) break;
              const uint32_t st = smem_u32(sm) + s * stage_bytes, bar = full_at + 8u * s;
              if (rank == 0 || !PAIR) mbar_arrive_expect_tx(full + s, bytes);
              if (p_t) {
                tma_load_3d<PAIR>(st, &job.p, at.p0, k, pz, bar);
                tma_load_3d<PAIR>(st + 64 * 128, &job.p, at.p0 + 64, k, pz, bar);
              } else {
                tma_load_3d<PAIR>(st, &job.p, k, at.p0, pz, bar);
              }
              if (q_t) {
                tma_load_3d<PAIR>(st + kPBytes, &job.q, at.q0, k, qz, bar);
                if (q_rows > 64) tma_load_3d<PAIR>(st + kPBytes + 64 * 128, &job.q, at.q0 + 64, k, qz, bar);
              } else {
                tma_load_3d<PAIR>(st + kPBytes, &job.q, k, at.q0, qz, bar);
              }
              turn = kProducers;
            }
            --turn;
            if (++s == stages) s = 0, ph ^= 1;
          }
        }
      };
      produce(jobs.job[0]);
      if (kTwo && jobs.count > 1) produce(jobs.job[1]);
      // Loads issued into shared memory land before the block can exit (a pair's leader counts
      // both CTAs' bytes).
      if (rank == 0 || !PAIR)
        for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j)
          drain_phase(full + j % stages, (j / stages) & 1, limit);
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
      const int64_t limit = jobs.job[0].d.wait_limit_ns;
      const auto multiply = [&](const ProductDev &p) {
        const int kblocks = blocks(p);
        const uint32_t p_step = desc_step(p.p_t), q_step = desc_step(p.q_t), idesc = p.idesc;
        const uint32_t p_first = desc_low(smem_u32(sm), p.p_t), q_first = desc_low(smem_u32(sm) + kPBytes, p.q_t);
        for (Walk walk(p, worker, workers); ok && walk.tile < p.tiles; walk.next()) {
          // A part of K shared by CTAs goes half into each accumulator, or evenly into several of 64
          // columns that are used once.
          const int seg_blocks = kApart ? (kblocks + p.segments - 1) / p.segments
                                 : SPLIT ? (kblocks + 1) / 2 : p.seg_blocks;
          for (int kb0 = 0; ok && kb0 < kblocks; kb0 += seg_blocks, ++unit) {
            const int kb1 = min(kb0 + seg_blocks, kblocks);
            const uint32_t acc = kApart ? unit : unit & 1, use = unit >> 1;
            if (!kApart && !(ok = wait_phase(acc_empty + acc, (use & 1) ^ 1, abort_flag, limit, p.status))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + acc * kAccCols;
            for (int kb = kb0; kb < kb1; ++kb) {
              if (!(ok = wait_phase(full + s, ph, abort_flag, limit, p.status))) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const uint32_t pd = p_first + s * (stage_bytes >> 4), qd = q_first + s * (stage_bytes >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f16<PAIR>(d, pd + k * p_step, qd + k * q_step, idesc, kb != kb0 || k != 0 ? 1u : 0u);
              commit<PAIR>(empty + s);
              if (++s == stages) s = 0, ph ^= 1;
            }
            if (ok && (!kApart || kb1 == kblocks)) commit<PAIR>(acc_full + (kApart ? 0 : acc));
          }
        }
      };
      if (one) {
        multiply(jobs.job[0].d);
        if (kTwo && jobs.count > 1) multiply(jobs.job[1].d);
      }
      if (one) commit<PAIR>(mma_done);
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const uint32_t acc_empty_at = PAIR ? map_to_rank(smem_u32(acc_empty), 0) : smem_u32(acc_empty);
    Shared w;
    w.arrived = arrived + (warp - 4) * kMaxAhead;
    w.acc_full = acc_full;
    w.tmem = tmem + ((uint32_t)(quad * 32) << 16);
    w.lane = lane;
    w.row0 = (PAIR ? rank * kP : 0) + quad * 32;
    w.abort_flag = abort_flag;
    w.unit = w.phases = 0;
    const auto release = [&](uint32_t acc) {
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(acc_empty_at + 8u * acc);
        else
          mbar_arrive(acc_empty + acc);
      }
    };
    bool ok = true;
    const auto drain_all = [&](const Job &job) {
      const ProductDev &p = job.d;
      const int qt = p.q_tile;
      const Walk start(p, worker, workers);
      if constexpr (!SPLIT) {
        if (SYMMETRIC || p.rows) {
          const int units = qt / kUnit, u0 = units * part / kPartsHere, u1 = units * (part + 1) / kPartsHere;
          w.buffers = smem_u32(sm) + stages * stage_bytes + (warp - 4) * jobs.warp_bytes;
          if constexpr (SEGMENTS)
            ok = move_tiles_of_segments<PAIR, NEWTON>(job, start, w, u0, u1, release);
          else
            ok = move_tiles<PAIR, SYMMETRIC, NEWTON>(job, start, w, u0, u1, release);
          return;
        }
      }
      if constexpr (!SYMMETRIC) {
        // This warp's 16-column chunks: a part of the tile's.
        const int c0 = qt / 16 * part / kPartsHere, chunks = qt / 16 * (part + 1) / kPartsHere - c0;
        if constexpr (SPLIT) {
          // The partial tile into shared memory (the stages: every MMA has read them).
          const bool two = !kApart && blocks(p) > 1;
          if (p.residual.p) {  // what is added in the end comes to L2 meanwhile: 0.7 us less
            const Tile t = tile_at<kTileP, SYMMETRIC>(p, worker);
            const int q_begin = qt * rank / splits, rows = qt * (rank + 1) / splits - q_begin;
            for (int i = warp - 4; i < 4 * rows; i += 4 * kPartsHere) {
              const int m = t.q0 + q_begin + (i >> 2), n = t.p0 + (i & 3) * 32 + lane;
              if ((lane & 7) == 0 && m < p.M && n < p.N)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(element(p.residual, t.z, m, n)));
            }
          }
          ok = warp_wait(acc_full, 0, abort_flag, p) && (!two || warp_wait(acc_full + 1, 0, abort_flag, p));
          if (!ok) return;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          float *mine = reinterpret_cast<float *>(sm) + c0 * 16 * kP + quad * 32 + lane;
          for (int c = 0; c < chunks; ++c) {
            uint32_t v[16], u[16];
            tmem_ld16(w.tmem + (c0 + c) * 16, v);
            if constexpr (kApart) {
              const int each = (blocks(p) + p.segments - 1) / p.segments;
              for (int k = 1; k * each < blocks(p); ++k) {
                tmem_ld16(w.tmem + k * kAccCols + (c0 + c) * 16, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
              }
            } else if (two) {
              tmem_ld16(w.tmem + kAccCols + (c0 + c) * 16, u);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mine[(c * 16 + i) * kP] = __uint_as_float(v[i]) + (two ? __uint_as_float(u[i]) : 0.f);
          }
        } else {
          constexpr int kMost = kAccCols / 16 / kPartsHere;
          for (Walk walk = start; ok && walk.tile < p.tiles; walk.next()) {
            const Tile t = tile_at<kTileP, false>(p, walk.tile);
            ok = drain_columns<kAccCols, kMost, SEGMENTS, NEWTON>(p, w, t.z, t.q0 + c0 * 16, t.p0 + w.row0 + lane,
                                                                  c0 * 16, chunks, release);
          }
        }
      }
    };
    drain_all(jobs.job[0]);
    if (kTwo && ok && jobs.count > 1) drain_all(jobs.job[1]);
  }

  if constexpr (SPLIT) {
    const ProductDev &p = jobs.job[0].d;
    const int qt = p.q_tile;
    // Each CTA adds a share of the tile's columns over the cluster, in rank order.
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();
    // A CTA that gave up has no partial tile.  A lane asks one of them: one after the other took 0.8 us.
    const bool gave_up =
        lane < splits && load_cluster(map_to_rank(smem_u32(const_cast<int *>(abort_flag)), lane)) != 0;
    const bool ok = !__any_sync(0xffffffffu, gave_up);
    const Tile t = tile_at<kTileP, SYMMETRIC>(p, worker);
    // A warp 32 neighbouring outputs of one row of out at a time.  Little code, as most launches run
    // through it once or twice and fetch it from far away.
    const int q_end = qt * (rank + 1) / splits, q_begin = qt * rank / splits;
    const uint32_t at0 = smem_u32(sm) + lane * 4;
#pragma unroll 1
    for (int i = warp; i < 4 * (q_end - q_begin); i += kThreadsHere / 32) {
      const int q = q_begin + (i >> 2), m = t.q0 + q, n = t.p0 + (i & 3) * 32 + lane;
      if (!ok || m >= p.M || n >= p.N) continue;
      const uint32_t at = at0 + (q * kP + (i & 3) * 32) * 4;
      float v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = r < splits ? __uint_as_float(load_cluster(map_to_rank(at, r))) : 0.f;
      const float bias = p.bias.p ? load_one(p.bias, 0, 0, n) : 0.f;
      const float residual =
          p.residual.p ? (NEWTON ? 1.f : p.residual_scale) * load_one(p.residual, t.z, m, n) : 0.f;
#pragma unroll
      for (int r = 1; r < 8; ++r) v[0] += v[r];
      finish_one<NEWTON>(p, t.z, m, n, p.scale * v[0], bias, residual);
    }
    cluster_sync();  // no CTA leaves while another may still read its part
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1 && lane == 0) drain_phase(mma_done, 0, jobs.job[0].d.wait_limit_ns);  // the MMAs ran
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

// A plane as a 3-D tiled map: boxes of 32 x 32 values.
bool make_plane_map(CUtensorMap *map, const PlaneDev &d, int64_t M, int64_t N, int64_t count) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const bool f32 = d.type == ENGRAM_DTYPE_F32;
  const int64_t bytes = f32 ? 4 : 2, stride = M > 1 ? d.stride * bytes : (N * bytes + 15) / 16 * 16;
  const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)(count > 1 ? d.batch * bytes : stride * M)};
  const cuuint32_t box[3] = {kUnit, 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, d.p, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceInfo {
  bool ready = false;
  int sms = 0, pairs = 0;  // pairs: CTA pairs that fit at once
  int clusters[9] = {};    // clusters of 2 .. 8 CTAs, two an SM, that do
};
DeviceInfo g_info[64];
std::mutex g_info_mu;

// Has the threads and the shared memory of a CTA that shares K.  Of a kernel with tensor memory the
// occupancy calls count one CTA an SM, whatever it takes; of this one the two that there are.
__global__ void __launch_bounds__(kSplitThreads, 2) two_an_sm_kernel() {}

using Kernel = void (*)(Jobs);
enum Form { kSingle, kSplit, kPair, kForms };
Kernel kernel_of(int form, int variant) {
  static constexpr Kernel all[kForms][kVariants] = {
      {product_kernel<false, false, kPlain>, product_kernel<false, false, kSegments>,
       product_kernel<false, false, kSymmetric>, product_kernel<false, false, kNewton>,
       product_kernel<false, false, kNewtonSegments>},
      {product_kernel<false, true, kPlain>, product_kernel<false, true, kSegments>, nullptr,
       product_kernel<false, true, kNewton>, nullptr},
      {product_kernel<true, false, kPlain>, product_kernel<true, false, kSegments>,
       product_kernel<true, false, kSymmetric>, product_kernel<true, false, kNewton>,
       product_kernel<true, false, kNewtonSegments>}};
  return all[form][variant];
}

cudaError_t device_info(DeviceInfo &out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_info_mu);
  DeviceInfo &d = g_info[dev & 63];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i = 0; i < kVariants * kForms && e == cudaSuccess; ++i)
      if (kernel_of(i / kVariants, i % kVariants))
        e = cudaFuncSetAttribute(kernel_of(i / kVariants, i % kVariants), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(i / kVariants == kSplit ? kSplitSmemBytes : kSmemBytes));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(d.sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&d.pairs, kernel_of(kPair, kPlain), &cfg)) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(two_an_sm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSplitSmemBytes);
    cfg.blockDim = dim3(kSplitThreads, 1, 1);
    cfg.dynamicSmemBytes = kSplitSmemBytes;
    for (int n = 2; n <= 8 && e == cudaSuccess; ++n) {
      attr.val.clusterDim.x = n;
      cfg.gridDim = dim3(2 * d.sms / n * n, 1, 1);
      e = cudaOccupancyMaxActiveClusters(d.clusters + n, two_an_sm_kernel, &cfg);
    }
    if (e != cudaSuccess) return e;
    d.ready = true;
  }
  out = d;
  return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of one matrix, `width` along P by qt along Q.
int64_t tiles_of(int64_t P, int64_t Q, int width, int qt, bool symmetric) {
  const int64_t tp = ceil_div(P, width), tq = ceil_div(Q, qt);
  if (!symmetric) return tp * tq;
  int64_t n = 0;
  for (int64_t i = 0; i < tp; ++i) {
    const int64_t end = P < (i + 1) * width ? P : (i + 1) * width, wide = (end - 1) / qt + 1;
    n += tq < wide ? tq : wide;
  }
  return n;
}

PlaneDev plane_of(const ProductParams &p, const Plane &x) {
  const int64_t step = x.type == ENGRAM_DTYPE_F32 ? 4 : 8;
  PlaneDev d{x.p, p.M > 1 ? x.stride : 0, p.count > 1 ? x.batch : 0, x.type, false};
  d.vec = ((uintptr_t)x.p & 15) == 0 && d.stride % step == 0 && d.batch % step == 0;
  return d;
}

// Bytes of a tiles' epilogue unit.
uint32_t unit_bytes(const PlaneDev &d) { return d.p ? 32 * kUnit * (d.type == ENGRAM_DTYPE_F32 ? 4 : 2) : 0; }

// A way to compute one product: its form, rows of out in the lanes or columns, the tile's width
// along Q, and what it is estimated to take in microseconds, less the launch's.
struct Plan {
  int form = kSingle, q_tile = 0, splits = 1;
  bool rows = false;
  double tile_us = 0, us = HUGE_VAL;  // tile_us: of one tile among others
  int64_t tiles = 0;
};

// What the choice goes by of a product.
struct Facts {
  ProductDev d;  // all but what a plan decides
  int64_t segment;  // most blocks of K in one accumulator
  bool tiles_epilogue;
};
Facts facts_of(const ProductParams &p) {
  Facts f{};
  ProductDev &d = f.d;
  d.out = plane_of(p, p.out);
  d.residual = plane_of(p, p.residual);
  d.pre = plane_of(p, p.pre);
  d.bias = plane_of(p, Plane{const_cast<void *>(p.bias), 0, 0, p.bias_type});
  d.act = p.act;
  d.scale = p.scale;
  d.residual_scale = p.residual_scale;
  d.status = p.status;
  d.diag_in = p.diag_in;
  d.diag_out = p.diag_out;
  d.diag_batch = p.diag_batch;
  d.diag_rows = p.diag_rows;
  d.diag_columns = p.diag_columns;
  d.diag_by = p.diag_by;
  d.diag_scale = p.diag_scale;
  d.wait_limit_ns = wait_limit_ns();
  d.M = (int32_t)p.M;
  d.N = (int32_t)p.N;
  d.many = p.count > 1;
  d.pass_blocks = (int32_t)ceil_div(p.K, kBK);
  d.kblocks = p.a_two ? 2 * d.pass_blocks : d.pass_blocks;
  // Segments as short as the output has the bits to show them; none of symmetric products.
  f.segment = p.out.type == ENGRAM_DTYPE_F32 || (p.pre.p && p.pre.type == ENGRAM_DTYPE_F32) ? kSegmentBlocks
              : p.symmetric                                                                 ? d.kblocks
                                                                                            : kHalfSegmentBlocks;
  d.seg_blocks = (int32_t)ceil_div(d.kblocks, ceil_div(d.kblocks, f.segment));
  d.segments = (int32_t)ceil_div(d.kblocks, d.seg_blocks);
  // The tiles' epilogue wants rows on 16-byte boundaries (a row that repeats has none apart).  Its
  // copies write whole 16 bytes, also where a row ends inside them: only the library's own planes,
  // which are fp16, have nothing there.  Storing such ends apart took the others 2 to 7 % longer.
  const auto reads = [&](const PlaneDev &x) { return !x.p || (x.vec && (p.M == 1 || x.stride >= p.N)); };
  const auto writes = [&](const PlaneDev &x) {
    return reads(x) && (!x.p || x.type == kTypeF16 || p.N % (x.type == ENGRAM_DTYPE_F32 ? 4 : 8) == 0);
  };
  f.tiles_epilogue = writes(d.out) && writes(d.pre) && reads(d.residual);
  return f;
}

// The estimates are fitted to every form at M 16 .. 32,768, N 64 .. 8192, K 64 .. 8192 (within 13 %
// on average; the form that they choose takes 2 % longer than the fastest).  A tile takes the
// longer of its products (by the stages of K, which single CTAs cannot take in faster than 0.17 us
// and pairs than 0.15) and of its epilogue (by the bytes that a value of out moves); the other of
// the two counts once, where nothing hides it.  No form reads the operands faster than memory gives
// them.
double read_us(const ProductParams &p, double of_b = 1) {
  return p.count * ((p.symmetric ? 0 : p.a_two ? 2 * p.M : p.M) + of_b * p.N) * p.K * 2 / 6.5e6;
}

// The best tile width of a form without splits.
Plan plan_form(const ProductParams &p, const Facts &f, int form, bool rows, const DeviceInfo &info) {
  const int64_t P = rows ? p.M : p.N, Q = rows ? p.N : p.M;
  const bool pair = form == kPair, q_t = (rows ? p.b : p.a).t;
  const int step = rows || pair ? kUnit : 16, workers = pair ? info.pairs : info.sms;
  Plan best;
  if (workers <= 0 || (pair && P <= kP)) return best;
  const double kb = f.d.kblocks, read = read_us(p);
  const auto bytes = [](const PlaneDev &x) { return !x.p ? 0 : x.type == ENGRAM_DTYPE_F32 ? 4 : 2; };
  const double moved = (1 + bytes(f.d.out) * (p.symmetric ? 2 : 1) + bytes(f.d.residual) + bytes(f.d.pre)) / 3.;
  for (int qt = pair ? kPairQMax : kQMax; qt >= step; qt -= step) {
    if (qt - step >= Q) continue;  // wider than Q
    Plan n;
    n.form = form;
    n.rows = rows;
    n.q_tile = qt;
    n.tiles = p.count * tiles_of(P, Q, pair ? 2 * kP : kP, qt, p.symmetric);
    const int staged = q_t ? (int)ceil_div(qt, pair ? 128 : 64) * (pair ? 128 : 64) : qt;
    double products, epilogue;
    if (pair) {
      products = kb * (rows ? 0.144 + 0.0005 * staged : fmax(0.157, 0.00106 * staged));
      epilogue = rows ? 1.3 + 0.0066 * qt * moved : 1.5 + 0.0104 * qt * moved;
    } else {
      products = kb * (rows ? 0.173 + 0.0004 * staged : 0.177);
      epilogue = rows ? 0.65 + 0.0058 * qt * moved : 0.9 + 0.0071 * qt * moved;
    }
    n.tile_us = fmax(products, epilogue);
    n.us = (pair ? 3.0 : 2.8) + fmax(ceil_div(n.tiles, workers) * n.tile_us, read) + fmin(products, epilogue);
    if (n.us < best.us) best = n;
  }
  return best;
}

// Accumulators of a CTA where n share K: two, or where K goes in segments one for each of its own.
int split_segments(const Facts &f, int n) {
  const int64_t own = ceil_div(ceil_div(f.d.kblocks, n), f.segment);
  return own > 2 ? (int)own : 2;
}

// K shared by 2 to 8 CTAs, two an SM: what a CTA takes of K, and the joining, by the rounds that its
// warps need for their share of the tile.  Only as many clusters as run at once: 36 of 8 take 11.8 us
// of 37 x 4608 x 4096, 37 of them 17.1 of 37 x 4736 x 4096.
Plan plan_split(const ProductParams &p, const Facts &f, const DeviceInfo &info) {
  Plan best;
  const double kb = f.d.kblocks;
  for (int qt = kQMax; qt >= 16; qt /= 2) {
    if (p.M <= qt / 2 && qt > 16) continue;
    const int width = p.M < qt ? (int)ceil_div(p.M, 16) * 16 : qt;
    const int64_t tiles = p.count * tiles_of(p.N, p.M, kP, width, p.symmetric);
    for (int n = 2; n <= 8; ++n) {
      if (tiles > info.clusters[n] || kb < n) continue;
      // Of fp32 outputs the accumulators of a part have to fit, and parts are not much longer than the
      // others' segments.
      if (split_segments(f, n) > (width <= kApartQMax && !p.newton ? (int)kSplitTmemCols / kApartQMax : 2)) continue;
      if (f.segment == kSegmentBlocks && f.d.segments > 1 && ceil_div(f.d.kblocks, n) > (n == 2 ? 24 : 32)) continue;
      Plan s;
      s.form = kSplit;
      s.q_tile = width;
      s.splits = n;
      s.tiles = tiles;
      // Stages at 0.2 us, of which reading b (a part again for each further tile of a) hides a part; or L2
      // gives no more than 16 TB/s.  Clusters of 3, 5, 6 and 7 lie less well on the SMs (20 x 4096 x
      // 4096: 4 9.3 us, 6 10.4, 8 9.3).
      const double stages = 0.2 * kb / n, read = read_us(p, 0.85 + 0.15 * ceil_div(p.M, width));
      const double taken = fmax(fmax(stages, read) + 0.4 * fmin(stages, read),
                                tiles * (kPBytes + 128. * width) / 16e6 * kb);
      s.us = 4.4 + 0.005 * width + taken + (n & (n - 1) ? 1.0 : 0.0) +
             0.45 * ceil_div(4 * ceil_div(width, n), kSplitThreads / 32);
      if (s.us < best.us) best = s;
    }
  }
  return best;
}

// Rows of out in the lanes where the tiles' epilogue can move it, and there are rows to fill them.
bool rows_of(const ProductParams &p, const Facts &f) { return f.tiles_epilogue && (p.symmetric || p.M > 64); }

Plan plan_of(const ProductParams &p, const Facts &f, const DeviceInfo &info) {
  const bool rows = rows_of(p, f);
  Plan best = plan_form(p, f, kSingle, rows, info);
  for (const Plan &n : {plan_form(p, f, kPair, rows, info), p.symmetric ? Plan() : plan_split(p, f, info)})
    if (n.us < best.us) best = n;
  return best;
}

// Bytes of a stage, and those that the stages of a plan should have at least: where K is short,
// moving out's values is the work, and buffers for them come first.
int64_t stage_bytes_of(const ProductParams &p, const Plan &plan) {
  const int staged = plan.form == kPair ? plan.q_tile / 2 : plan.q_tile;
  return kPBytes + ((plan.rows ? p.b : p.a).t ? (staged + 63) / 64 * 64 : staged) * 128;
}
int64_t reserve_of(const ProductParams &p, int64_t stage) {
  return (p.K <= 4 * kBK ? kProducers : 5) * stage;
}

// A job of a plan; its share of the shared memory (the epilogue's buffers) in `buffers`, which leave
// `reserve` bytes for stages.
cudaError_t job_of(const ProductParams &p, const Facts &f, const Plan &plan, int64_t reserve, bool segments, Job &job,
                   int64_t &buffers) {
  const Operand &op = plan.rows ? p.a : p.b, &oq = plan.rows ? p.b : p.a;
  const int64_t P = plan.rows ? p.M : p.N, Q = plan.rows ? p.N : p.M;
  ProductDev &d = job.d;
  d = f.d;
  d.rows = plan.rows;
  d.p_next = p.a_two && plan.rows;
  d.q_next = p.a_two && !plan.rows;
  d.p_t = op.t;
  d.q_t = oq.t;
  d.q_tile = plan.q_tile;
  const int q_staged = plan.form == kPair ? plan.q_tile / 2 : plan.q_tile;
  d.q_rows = (int32_t)((stage_bytes_of(p, plan) - kPBytes) / 128);
  const int warps = 4 * (plan.form == kPair ? kPairParts : kParts);
  buffers = 0;
  if (plan.rows) {
    // One buffer of each sort at least.
    d.ahead_bytes = unit_bytes(d.residual);
    d.slot_bytes = unit_bytes(d.out) > unit_bytes(d.pre) ? unit_bytes(d.out) : unit_bytes(d.pre);
    d.ahead = d.ahead_bytes ? 1 : 0;
    d.slots = 1;
    const auto bytes = [&](int ahead, int slots) {
      return (int64_t)warps * (ahead * d.ahead_bytes + slots * d.slot_bytes);
    };
    // With sums in segments one buffer serves both where it can.
    if (segments && d.ahead && !d.pre.p && d.ahead_bytes == d.slot_bytes) d.slots = 0;
    const int64_t most = segments ? 0 : kBudget - reserve;
    if (bytes(d.ahead, 2) <= most) d.slots = 2;
    while (d.ahead && d.ahead < kMaxAhead && bytes(d.ahead + 1, d.slots) <= most) ++d.ahead;
    buffers = bytes(d.ahead, d.slots);
  }
  if (plan.form == kSplit) d.segments = split_segments(f, plan.splits);
  const int width = plan.form == kPair ? 2 * kP : kP;
  const int64_t matrix_tiles = tiles_of(P, Q, width, plan.q_tile, p.symmetric), tiles = matrix_tiles * p.count;
  if (tiles > INT32_MAX / 16) return cudaErrorInvalidConfiguration;  // group_tiles stay in 31 bits too
  d.tiles_p = (int32_t)ceil_div(P, width);
  d.tiles_q = (int32_t)ceil_div(Q, plan.q_tile);
  d.matrix_tiles = (int32_t)matrix_tiles;
  d.tiles = (int32_t)tiles;
  if (!p.symmetric) {
    // b's slices of a group, about 32 MB, stay in L2 while a's pass by (65,536 x 4096 x 6144 in groups
    // of 8 columns of tiles 1925 us, of 16 1979; 16,384 x 6144 x 4096 493 and 476).
    const int64_t columns = plan.rows ? d.tiles_q : d.tiles_p, rows = plan.rows ? d.tiles_p : d.tiles_q;
    const int64_t slice = (plan.rows ? plan.q_tile : width) * p.K * 2;
    int64_t most = (32 << 20) / slice;
    most = most < 4 ? 4 : most > 16 ? 16 : most;
    const int64_t groups = ceil_div(columns, most), per = ceil_div(columns, groups);
    d.group_columns = (int32_t)per;
    d.group_tiles = (int32_t)(per * rows);
    d.last_columns = (int32_t)(columns - columns / per * per);
    d.by_matrix = fast_div_of((uint32_t)matrix_tiles);
    d.by_group = fast_div_of((uint32_t)d.group_tiles);
    d.by_columns = fast_div_of((uint32_t)per);
    d.by_last = fast_div_of(d.last_columns ? (uint32_t)d.last_columns : 1);
  } else {
    d.by_matrix = fast_div_of((uint32_t)matrix_tiles);
  }
  // kind::f16: fp32 accumulator, the operands' type (0: f16, 1: bf16), which of them are MN-major.
  d.idesc = 1u << 4 | (p.f16 ? 0u : 1u << 7 | 1u << 10) | (uint32_t)d.p_t << 15 | (uint32_t)d.q_t << 16 |
            (uint32_t)(plan.q_tile >> 3) << 17 | (uint32_t)(width >> 4) << 24;
  const bool ok = make_map(&job.p, op, P, p.K, p.count + d.p_next, kP) &&
                  make_map(&job.q, oq, Q, p.K, p.count + d.q_next, (uint32_t)q_staged) &&
                  (!plan.rows || (make_plane_map(&job.out, d.out, p.M, p.N, p.count) &&
                                  (!d.pre.p || make_plane_map(&job.pre, d.pre, p.M, p.N, p.count)) &&
                                  (!d.residual.p || make_plane_map(&job.residual, d.residual, p.M, p.N, p.count))));
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}

// Launches the jobs of plans of one form; buffers: the most that one of them has for its epilogue.
cudaError_t launch_jobs(Jobs &jobs, const Plan &plan, int64_t buffers, int variant, const DeviceInfo &info,
                        cudaStream_t stream) {
  jobs.job[0].d.withhold = take_withheld_launch();
  jobs.splits = plan.splits;
  jobs.warp_bytes = (uint32_t)(buffers / (4 * (plan.form == kPair ? kPairParts : kParts)));
  int64_t tiles = 0;
  for (int i = 0; i < jobs.count; ++i) {
    const uint32_t bytes = kPBytes + jobs.job[i].d.q_rows * 128;
    if (bytes > jobs.stage_bytes) jobs.stage_bytes = bytes;
    tiles += jobs.job[i].d.tiles;
  }
  jobs.stages = (int32_t)(((plan.form == kSplit ? kSplitBudget : kBudget) - (plan.form == kSplit ? 0 : buffers)) /
                          jobs.stage_bytes);
  if (jobs.stages > kMaxStages) jobs.stages = kMaxStages;
  if (jobs.stages < kProducers) return cudaErrorInvalidConfiguration;
  if (plan.form == kSplit && variant != kNewton) variant = jobs.job[0].d.segments > 2 ? kSegments : kPlain;
  const Kernel kernel = kernel_of(plan.form, variant);
  if (plan.form == kPair)
    return launch(kernel, 2 * (tiles < info.pairs ? tiles : info.pairs), kPairThreads, kSmemBytes, stream, 2, jobs);
  if (plan.form == kSplit)
    return launch(kernel, tiles * plan.splits, kSplitThreads, kSplitSmemBytes, stream, plan.splits, jobs);
  return launch(kernel, tiles < info.sms ? tiles : info.sms, kThreads, kSmemBytes, stream, 1, jobs);
}

}  // namespace

cudaError_t launch_product(const ProductParams &p, cudaStream_t stream) {
  if (few_rows_supported(p)) return launch_few_rows(p, stream);
  DeviceInfo info;
  cudaError_t e = device_info(info);
  if (e != cudaSuccess) return e;
  const Facts f = facts_of(p);
  const Plan plan = plan_of(p, f, info);
  if (p.symmetric) {  // half of the tiles, unless that many run side by side in any case, or K is long
    ProductParams whole = p;
    whole.symmetric = false;
    if (f.d.kblocks > kHalfSegmentBlocks || plan_of(whole, facts_of(whole), info).us <= plan.us)
      return launch_product(whole, stream);
  }
  Jobs jobs{};
  jobs.count = 1;
  int64_t buffers;
  const int64_t reserve = reserve_of(p, stage_bytes_of(p, plan));
  if ((e = job_of(p, f, plan, reserve, f.d.segments > 1, jobs.job[0], buffers)) != cudaSuccess) return e;
  const bool segments = f.d.segments > 1 && plan.form != kSplit;
  const int variant = p.symmetric ? kSymmetric
                      : p.newton  ? segments ? kNewtonSegments : kNewton
                                  : segments ? kSegments : kPlain;
  return launch_jobs(jobs, plan, buffers, variant, info, stream);
}

cudaError_t launch_products(const ProductParams &p0, const ProductParams &p1, cudaStream_t stream) {
  DeviceInfo info;
  cudaError_t e = device_info(info);
  if (e != cudaSuccess) return e;
  const ProductParams *p[2] = {&p0, &p1};
  const Facts f[2] = {facts_of(p0), facts_of(p1)};
  Plan alone[2], best[2];
  for (int i = 0; i < 2; ++i) alone[i] = plan_of(*p[i], f[i], info);
  if (few_rows_supported(p0) || few_rows_supported(p1)) {
    if ((e = launch_product(p0, stream)) != cudaSuccess) return e;
    return launch_product(p1, stream);
  }
  // Together in one launch, both in one form, the one of the longer tiles first: its last wave is
  // filled by the other's tiles.  Another launch takes 2.5 us.
  double us = alone[0].us + alone[1].us + 2.5;
  bool together = false;
  for (int form : {kSingle, kPair}) {
    Plan n[2];
    for (int i = 0; i < 2; ++i) n[i] = plan_form(*p[i], f[i], form, rows_of(*p[i], f[i]), info);
    if (n[0].us == HUGE_VAL || n[1].us == HUGE_VAL) continue;
    const int workers = form == kPair ? info.pairs : info.sms;
    const double work = (n[0].tiles * n[0].tile_us + n[1].tiles * n[1].tile_us) / workers;
    const double longest = fmax(n[0].tile_us, n[1].tile_us), shorter = fmin(n[0].tile_us, n[1].tile_us);
    const double rest = fmin(n[0].us - n[0].tile_us, n[1].us - n[1].tile_us);  // what counts once
    const double both = fmin(rest, 5.) + fmax(longest, work + 0.5 * shorter);
    if (both < us) us = both, best[0] = n[0], best[1] = n[1], together = true;
  }
  if (!together) {
    if ((e = launch_product(p0, stream)) != cudaSuccess) return e;
    return launch_product(p1, stream);
  }
  const int a = best[0].tile_us >= best[1].tile_us ? 0 : 1, b = 1 - a;
  Jobs jobs{};
  jobs.count = 2;
  const bool segments = f[0].d.segments > 1 || f[1].d.segments > 1;
  int64_t buffers[2], stage = 0, reserve = 0;
  for (int i = 0; i < 2; ++i)
    if (stage_bytes_of(*p[i], best[i]) > stage) stage = stage_bytes_of(*p[i], best[i]);
  for (int i = 0; i < 2; ++i)
    if (reserve_of(*p[i], stage) > reserve) reserve = reserve_of(*p[i], stage);
  if ((e = job_of(*p[a], f[a], best[a], reserve, segments, jobs.job[0], buffers[0])) != cudaSuccess) return e;
  if ((e = job_of(*p[b], f[b], best[b], reserve, segments, jobs.job[1], buffers[1])) != cudaSuccess) return e;
  const int64_t most = best[0].form == kPair ? info.pairs : info.sms, tiles = best[0].tiles + best[1].tiles;
  const int64_t workers = tiles < most ? tiles : most;
  ProductDev &second = jobs.job[1].d;
  second.shift = (int32_t)(best[a].tiles % workers);
  const int64_t lights = workers - second.shift;
  int64_t extra = second.shift ? (int64_t)(best[a].tile_us / best[b].tile_us) : 0;
  if (extra > best[b].tiles / lights) extra = best[b].tiles / lights;
  second.extra = (int32_t)extra;
  return launch_jobs(jobs, best[0], buffers[0] > buffers[1] ? buffers[0] : buffers[1],
                     segments ? kSegments : kPlain, info, stream);
}

}  // namespace engram

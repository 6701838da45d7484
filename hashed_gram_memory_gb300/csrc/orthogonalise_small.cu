// orthogonalise_small.cu -- engram_orthogonalise for matrices whose shorter side is at most 128:
// the whole iteration in one launch, a cluster of 1 to 8 CTAs a matrix.
//
// Each CTA keeps its columns of X (the shorter side padded to 128 rows) in shared memory from the
// first step to the last, in blocks of 128 rows x 64 columns with the 128-byte swizzle.  One and the
// same block is a K-major operand of X X^T (rows along K = its columns) and an MN-major operand of
// B X (its columns along the instruction's N, its rows along K), so nothing is ever transposed:
//   A    = sum over the CTAs of X_c X_c^T: tensor cores, the parts added through distributed
//          shared memory in rank order, the fp16 result written to every CTA;
//   B    = b A + c A^2: every CTA by itself;
//   X_c  = a X_c + B X_c: every CTA its columns, in place.
// All threads but the one that issues the instructions serve the epilogues, lanes being rows.
//
// What is rounded, and where, and the diagonals that stay fp32 are as in orthogonalise.cu (16 x 700: 1.9e-3
// off with its own rounding to bf16, 2.4e-3 with the diagonals rounded, which takes 128 x 128 1.2 us
// less).  Bound by the latency of a step, 2.5 us in a CTA by itself and 6 where two join A; fp32 with
// momentum, in us, beside the chain of launches:
//   1 of  64 x   64   19 and 63        32 of  64 x  256    29 and  76
//   1 of 128 x  128   25 and 60        16 of 128 x 1024    56 and  92
//   1 of 128 x  512   51 and 68      1000 of 128 x  128   188 and 303
//   1 of 100 x 3500   80 and 80       300 of 128 x  896   328 and 428
#include <stddef.h>

#include <mutex>

#include "launch.cuh"
#include "tensor_pieces.cuh"
#include "train_internal.cuh"
#include "values.cuh"

namespace engram {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kR = 128;                      // rows
constexpr int kMostBlocks = 7;               // of 64 columns a CTA
constexpr uint32_t kBlock = kR * 64 * 2;     // bytes
constexpr int kPitch = kR + 4;               // floats between rows of a part of A: no bank conflicts
constexpr uint32_t kSquare = 2 * kBlock;     // A or B
constexpr uint32_t kPart = kR * kPitch * 4;  // fp32 A; B lies in the same place later
constexpr float kHeld = 256.f;               // what fp16 values are held times
static_assert(kPart >= kSquare);
constexpr size_t smem_bytes(int blocks) { return 1024 + (size_t)blocks * kBlock + kSquare + kPart; }
static_assert(smem_bytes(kMostBlocks) + 1024 <= 227 * 1024);
// A CTA takes all of an SM's TMEM.  One of a cluster (4 blocks and more) leaves no shared memory for
// a CTA of another launch that holds TMEM, a split product's with 100 KB and more: two clusters on
// two SMs, each with the TMEM that the other wants, would wait for ever.
static_assert(smem_bytes(kMostBlocks / 2 + 1) + 100 * 1024 > 228 * 1024);

struct SmallDev {
  Plane g, momentum, out;
  int32_t *status;
  int64_t wait_limit_ns;
  int32_t r, w, blocks, cluster, steps;  // the sides; 64-column blocks a CTA
  float beta, eps, scale, a, b, c;
  bool tall, nesterov, wide_out;  // wide_out: rows of out on 16 bytes
  bool withhold;  // test hook: a cluster's first CTA waits for an arrival that never comes
};

constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;  // groups of 8 rows, version 1, SWIZZLE_128B

// fp16 operands, fp32 accumulator; q_t: Q is MN-major.
__device__ __forceinline__ uint32_t idesc_of(int n, bool q_t) {
  return 1u << 4 | (uint32_t)q_t << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(kR >> 4) << 24;
}
__device__ __forceinline__ void umma(uint32_t d, uint32_t p_low, uint32_t q_low, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(p_low), "r"(q_low), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
      : "memory");
}
// The low half of a descriptor: the address, and the stride between blocks along the rows (MN-major).
__device__ __forceinline__ uint32_t low_of(uint32_t addr, uint32_t between) {
  return ((addr >> 4) & 0x3FFF) | (between >> 4) << 16;
}

// Where 16-byte piece `piece` of row i of a block lies.
__device__ __forceinline__ uint32_t at(uint32_t block, int i, int piece) {
  return block + i * 128 + ((piece ^ (i & 7)) << 4);
}
__device__ __forceinline__ uint4 ld16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void st16(uint32_t a, const uint4 &v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t halves(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t bfloats(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 floats(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

// Value i of 16 (a chain of 16 selections takes 0.1 us longer a time).
__device__ __forceinline__ float pick(const uint32_t (&v)[16], int i) {
  uint32_t a[8], b[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = i & 1 ? v[2 * k + 1] : v[2 * k];
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = i & 2 ? a[2 * k + 1] : a[2 * k];
  const uint32_t lo = i & 4 ? b[1] : b[0], hi = i & 4 ? b[3] : b[2];
  return __uint_as_float(i & 8 ? hi : lo);
}
// Zero at row i, column i of a square matrix, after the row was stored.
__device__ __forceinline__ void clear_diagonal(uint32_t square, int i) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at(square + (i >> 6) * kBlock, i, (i & 63) >> 3) + (i & 7) * 2),
               "h"((uint16_t)0)
               : "memory");
}

// f(row of X, column of X of this CTA, u) over the CTA's elements; with FIRST the momentum moves.
// Neighbouring threads take neighbouring elements of a matrix row in memory; a warp 128 of each of
// kRows rows at a time: all of their loads, then the rest.
constexpr int kRows = 4;
template <bool FIRST, typename T, typename F>
__device__ __forceinline__ void over_elements(const SmallDev &p, int64_t z, int col0, int columns, F f) {
  const int fast = p.tall ? p.r : columns, slow = p.tall ? columns : p.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m0 = p.tall ? col0 : 0, n0 = p.tall ? 0 : col0;  // where the CTA's share begins
  for (int s = warp; s < slow; s += kRows * kWarps) {
    const T *g[kRows];
    float *m[kRows] = {};
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      g[k] = static_cast<const T *>(p.g.p) + z * p.g.batch + (m0 + s + k * kWarps) * p.g.stride + n0 + lane;
      if (p.momentum.p)
        m[k] = static_cast<float *>(p.momentum.p) + z * p.momentum.batch + (m0 + s + k * kWarps) * p.momentum.stride +
               n0 + lane;
    }
    for (int q0 = 0; q0 < fast; q0 += 128) {
      float u[kRows][4], v[kRows][4];
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[k][i] = q0 + 32 * i + lane < fast && s + k * kWarps < slow ? to_float(__ldg(g[k] + q0 + 32 * i)) : 0.f;
      if (p.momentum.p) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[k][i] = q0 + 32 * i + lane < fast && s + k * kWarps < slow ? m[k][q0 + 32 * i] : 0.f;
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FIRST) {
              v[k][i] = fmaf(p.beta, v[k][i], u[k][i]);
              if (q0 + 32 * i + lane < fast && s + k * kWarps < slow) m[k][q0 + 32 * i] = v[k][i];
            }
            u[k][i] = p.nesterov ? fmaf(p.beta, v[k][i], u[k][i]) : v[k][i];
          }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q0 + 32 * i + lane < fast && s + k * kWarps < slow)
            p.tall ? f(q0 + 32 * i + lane, s + k * kWarps, u[k][i]) : f(s + k * kWarps, q0 + 32 * i + lane, u[k][i]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) orthogonalise_small_kernel(const __grid_constant__ SmallDev p) {
  extern __shared__ uint8_t sm_raw[];
  __shared__ uint64_t done, drained;  // the instructions issued have completed
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, gave_up;
  __shared__ Squares warp_sums[kWarps], cta_sum;
  __shared__ __align__(16) float diag_a[kR], diag_b[kR];
  uint8_t *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  const uint32_t X = smem_u32(sm), A = X + p.blocks * kBlock, B = A + kSquare, part = B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, share = warp >> 2;  // of the lanes, of the columns
  const int row = quad * 32 + lane;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
  const int64_t z = blockIdx.x / p.cluster;
  const int col0 = rank * p.blocks * 64, columns = max(0, min(p.blocks * 64, p.w - col0));

  if (threadIdx.x == 0) {
    mbar_init(&done, p.withhold && rank == 0 ? 2 : 1);
    mbar_init(&drained, 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The padding of X is zero.
  for (uint32_t i = threadIdx.x * 16; i < p.blocks * kBlock; i += kThreads * 16) st16(X + i, make_uint4(0, 0, 0, 0));
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot, quad_tmem = tmem + ((uint32_t)(quad * 32) << 16);
  dependency_wait();

  const auto together = [&] {
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
  };

  // The momentum step, the norm, X.
  Squares sum{};
  over_elements<true, T>(p, z, col0, columns, [&](int, int, float u) { sum.add(u); });
  for (int i = 16; i > 0; i >>= 1) sum.add(sum.across_lane(i));
  if (lane == 0) warp_sums[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    Squares s{};
    for (int i = 0; i < kWarps; ++i) s.add(warp_sums[i]);
    cta_sum = s;
  }
  together();
  sum = cta_sum;
  if (p.cluster > 1) {
    sum = Squares{};
    for (int r = 0; r < p.cluster; ++r) {
      const uint32_t from = map_to_rank(smem_u32(&cta_sum), r);
      Squares s{};
      s.plain = __uint_as_float(load_cluster(from + offsetof(Squares, plain)));
      s.small = __uint_as_float(load_cluster(from + offsetof(Squares, small)));
      s.large = __uint_as_float(load_cluster(from + offsetof(Squares, large)));
      sum.add(s);
    }
  }
  const Norm norm(sum, p.eps, kHeld);
  over_elements<false, T>(p, z, col0, columns, [&](int i, int j, float u) {
    const __half v = __float2half_rn(u * norm.first * norm.second);
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at(X + (j >> 6) * kBlock, i, (j & 63) >> 3) + (j & 7) * 2),
                 "h"(__half_as_ushort(v))
                 : "memory");
  });

  uint32_t phase = 0;
  // The same in every lane of a warp, and after run's barrier in every warp.  Once it is false a CTA
  // issues nothing more and touches neither its matrices nor tensor memory, which instructions may
  // still be reading and writing; it only meets the others of its cluster.
  bool ok = true;
  // What the generic proxy has written is there for the tensor cores; then one thread issues.
  const auto run = [&](auto issue) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    ok = __syncthreads_and(ok);
    if (!ok) return;
    if (threadIdx.x == 0) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      issue();
      umma_commit(&done);
    }
    __syncwarp();
    ok = __all_sync(0xffffffffu, wait_phase(&done, phase, &abort_flag, p.wait_limit_ns, p.status));
    phase ^= 1;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  };
  const int c0 = share * 32;  // of 128 columns of A and B
  __nv_bfloat16 *const out = static_cast<__nv_bfloat16 *>(p.out.p) + z * p.out.batch;

  for (int step = 0; step < p.steps; ++step) {
    // ---- A
    run([&] {
      const uint32_t x = low_of(X, 16), idesc = idesc_of(kR, false);
      for (int k = 0; k < p.blocks; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          umma(tmem, x + k * (kBlock >> 4) + 2 * i, x + k * (kBlock >> 4) + 2 * i, idesc, k + i > 0);
    });
    if (ok) {
      uint32_t v[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncwarp();
        tmem_ld16(quad_tmem + c0 + 16 * h, v);
        if (p.cluster == 1) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = halves(__uint_as_float(v[8 * q + 2 * i]) / kHeld, __uint_as_float(v[8 * q + 2 * i + 1]) / kHeld);
            const int c = c0 + 16 * h + 8 * q;
            st16(at(A + (c >> 6) * kBlock, row, (c & 63) >> 3), make_uint4(w[0], w[1], w[2], w[3]));
          }
          if (quad == share) {
            const float d = pick(v, lane & 15) / (kHeld * kHeld);
            if (lane >> 4 == h) {
              diag_a[row] = d;
              clear_diagonal(A, row);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st16(part + (row * kPitch + c0 + 16 * h + 4 * q) * 4,
                 make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
        }
      }
    }
    if (p.cluster > 1) {
      cluster_sync();
      // A share of the rows each, added in rank order and written to all.
      const int rows = kR / p.cluster, r0 = rank * rows;
      for (int i = threadIdx.x; ok && i < rows * 32; i += kThreads) {
        const int r = r0 + (i >> 5), c = (i & 31) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          v[q] = q < p.cluster ? load4_cluster(map_to_rank(part + (r * kPitch + c) * 4, q)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 8; ++q) s.x += v[q].x, s.y += v[q].y, s.z += v[q].z, s.w += v[q].w;
        // A warp has a row: the lane of its diagonal takes it out, a lane for each CTA hands it on.
        const int k = r & 3;
        const bool here = r >> 2 == c >> 2;
        const float d = __shfl_sync(0xffffffffu, k == 0 ? s.x : k == 1 ? s.y : k == 2 ? s.z : s.w, r >> 2);
        s = make_float4(here && k == 0 ? 0.f : s.x, here && k == 1 ? 0.f : s.y, here && k == 2 ? 0.f : s.z,
                        here && k == 3 ? 0.f : s.w);
        if (lane < p.cluster)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(diag_a + r), lane)),
                       "f"(d / (kHeld * kHeld))
                       : "memory");
        const uint32_t lo = halves(s.x / kHeld, s.y / kHeld), hi = halves(s.z / kHeld, s.w / kHeld);
        const uint32_t to = at(A + (c >> 6) * kBlock, r, (c & 63) >> 3) + (c & 4) * 2;
        for (int q = 0; q < p.cluster; ++q)
          asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(map_to_rank(to, q)), "r"(lo), "r"(hi)
                       : "memory");
      }
      cluster_sync();
    }
    // ---- B
    run([&] {
      const uint32_t x = low_of(A, 16), idesc = idesc_of(kR, false);
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          umma(tmem + kR, x + k * (kBlock >> 4) + 2 * i, x + k * (kBlock >> 4) + 2 * i, idesc, k + i > 0);
    });
    const float d = diag_a[row], mine = fmaf(p.c, d, p.b);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!ok) break;
      uint32_t v[16];
      __syncwarp();
      tmem_ld16(quad_tmem + kR + c0 + 16 * h, v);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = c0 + 16 * h + 8 * q;
        const uint32_t to = at((c >> 6) * kBlock, row, (c & 63) >> 3);
        const uint4 have = ld16(A + to);
        const float4 e0 = *reinterpret_cast<const float4 *>(diag_a + c), e1 = *reinterpret_cast<const float4 *>(diag_a + c + 4);
        const uint32_t w[4] = {have.x, have.y, have.z, have.w};
        const float e[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = floats(w[i]);
          y[i] = halves(fmaf(fmaf(p.c, e[2 * i], mine), f.x, p.c / kHeld * __uint_as_float(v[8 * q + 2 * i])),
                        fmaf(fmaf(p.c, e[2 * i + 1], mine), f.y, p.c / kHeld * __uint_as_float(v[8 * q + 2 * i + 1])));
        }
        st16(B + to, make_uint4(y[0], y[1], y[2], y[3]));
      }
      if (quad == share) {
        const float e = fmaf(mine, d, p.c / (kHeld * kHeld) * pick(v, lane & 15));
        if (lane >> 4 == h) {
          diag_b[row] = e;
          clear_diagonal(B, row);
        }
      }
    }
    // ---- X
    run([&] {
      const uint32_t b = low_of(B, 16);
      for (int n = 0; n < p.blocks; n += 4) {
        const int wide = min(4, p.blocks - n) * 64;
        const uint32_t x = low_of(X + n * kBlock, kBlock), idesc = idesc_of(wide, true);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 rows of X: 2048 bytes
          umma(tmem + n * 64, b + (k >> 2) * (kBlock >> 4) + 2 * (k & 3), x + k * (2048 >> 4), idesc, k > 0);
      }
    });
    const float own = p.a + diag_b[row];
    const bool last = step == p.steps - 1;
    if (last) {  // out is written by all of a matrix's CTAs or by none
      ok = __syncthreads_and(ok);
      if (p.cluster > 1) {
        if (threadIdx.x == 0) gave_up = !ok;
        cluster_sync();
        const uint32_t flag = smem_u32(&gave_up);
        ok = !__any_sync(0xffffffffu, lane < p.cluster && load_cluster(map_to_rank(flag, lane)) != 0);
      }
    }
    for (int c = share * 16; ok && c < p.blocks * 64; c += kWarps / 4 * 16) {
      uint32_t v[16];
      __syncwarp();
      tmem_ld16(quad_tmem + c, v);
      float x[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t to = at(X + (c >> 6) * kBlock, row, ((c & 63) >> 3) + q);
        const uint4 have = ld16(to);
        const uint32_t w[4] = {have.x, have.y, have.z, have.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = floats(w[i]);
          x[8 * q + 2 * i] = fmaf(own, f.x, __uint_as_float(v[8 * q + 2 * i]) / kHeld);
          x[8 * q + 2 * i + 1] = fmaf(own, f.y, __uint_as_float(v[8 * q + 2 * i + 1]) / kHeld);
        }
        if (last && !p.tall) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[8 * q + i] *= p.scale / kHeld;
          st16(to, make_uint4(bfloats(x[8 * q], x[8 * q + 1]), bfloats(x[8 * q + 2], x[8 * q + 3]),
                              bfloats(x[8 * q + 4], x[8 * q + 5]), bfloats(x[8 * q + 6], x[8 * q + 7])));
        } else if (!last) {
          st16(to, make_uint4(halves(x[8 * q], x[8 * q + 1]), halves(x[8 * q + 2], x[8 * q + 3]),
                              halves(x[8 * q + 4], x[8 * q + 5]), halves(x[8 * q + 6], x[8 * q + 7])));
        }
      }
      if (last && p.tall && row < p.r)  // a warp's lanes are neighbours in memory
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < columns) from_float(out[(col0 + c + i) * p.out.stride + row], x[i] * (p.scale / kHeld));
    }
  }
  // A wide matrix leaves by rows: straight from the lanes, 2 bytes of a row each, 128 x 128 took 18 us.
  if (!p.tall) {
    __syncthreads();
    if (ok)
      for (int i = warp; i < p.r; i += kWarps) {
        __nv_bfloat16 *to = out + i * p.out.stride + col0;
        if (p.wide_out) {
          for (int q = lane; q * 8 < columns; q += 32) {
            const uint4 v = ld16(at(X + (q >> 3) * kBlock, i, q & 7));
            if (q * 8 + 8 <= columns) {
              *reinterpret_cast<uint4 *>(to + q * 8) = v;
            } else {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (q * 8 + k < columns)
                  reinterpret_cast<uint16_t *>(to)[q * 8 + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
            }
          }
        } else {
          for (int j = lane; j < columns; j += 32) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(v)
                         : "r"(at(X + (j >> 6) * kBlock, i, (j & 63) >> 3) + (j & 7) * 2)
                         : "memory");
            reinterpret_cast<uint16_t *>(to)[j] = v;
          }
        }
      }
  }

  // ---- teardown
  // After a wait that gave up: the instructions issued end before the memory that they use goes.
  if (threadIdx.x == 0 && abort_flag) {
    umma_commit(&drained);
    drain_phase(&drained, 0, p.wait_limit_ns);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  together();  // no CTA leaves while another may still read or write its memory
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

std::mutex g_mu;
bool g_ready[64];

}  // namespace

namespace {
// CTAs a matrix, as few as hold it: what joining A takes is more than what it saves.
int cluster_of(int64_t w) {
  int cluster = 1;
  while (cluster * kMostBlocks * 64 < w) cluster *= 2;
  return cluster;
}
}  // namespace

// Clusters of 4 and 8 spend more on joining A than on products.  They win while every matrix has its
// CTAs at once; where there are more the chain, whose products share no A, is ahead: 300 of
// 100 x 1800 1259 us here and 755 there, 500 of 16 x 2000 1813 and 807.
bool orthogonalise_small_supported(const OrthogonaliseParams &p) {
  const int64_t r = p.M < p.N ? p.M : p.N, w = p.M < p.N ? p.N : p.M;
  if (r > kR || w > 8 * kMostBlocks * 64) return false;
  const int cluster = cluster_of(w);
  return cluster <= 2 || p.count * cluster <= kSms;
}

cudaError_t launch_orthogonalise_small(const OrthogonaliseParams &p, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ready[dev & 63]) {
      constexpr auto attribute = cudaFuncAttributeMaxDynamicSharedMemorySize;
      e = cudaFuncSetAttribute(orthogonalise_small_kernel<float>, attribute, (int)smem_bytes(kMostBlocks));
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(orthogonalise_small_kernel<__nv_bfloat16>, attribute, (int)smem_bytes(kMostBlocks));
      if (e != cudaSuccess) return e;
      g_ready[dev & 63] = true;
    }
  }
  SmallDev d{};
  d.g = p.g;
  d.momentum = p.momentum;
  d.out = p.out;
  d.status = p.status;
  d.wait_limit_ns = wait_limit_ns();
  d.tall = p.M > p.N;
  d.r = (int32_t)(d.tall ? p.N : p.M);
  d.w = (int32_t)(d.tall ? p.M : p.N);
  d.steps = p.steps;
  d.beta = p.beta;
  d.eps = p.eps;
  d.scale = p.scale;
  d.a = p.a;
  d.b = p.b;
  d.c = p.c;
  d.nesterov = p.nesterov;
  d.wide_out = reinterpret_cast<uintptr_t>(p.out.p) % 16 == 0 && p.out.stride % 8 == 0 &&
               (p.count == 1 || p.out.batch % 8 == 0);
  d.withhold = take_withheld_launch();
  const int blocks = (d.w + 63) / 64;
  d.cluster = cluster_of(d.w);
  d.blocks = (blocks + d.cluster - 1) / d.cluster;
  const auto kernel = p.g.type == ENGRAM_DTYPE_F32 ? orthogonalise_small_kernel<float>
                                                   : orthogonalise_small_kernel<__nv_bfloat16>;
  return launch(kernel, p.count * d.cluster, kThreads, smem_bytes(d.blocks), stream, d.cluster, d);
}

}  // namespace engram

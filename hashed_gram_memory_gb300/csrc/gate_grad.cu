// gate_grad.cu -- the backward pass of the gated add (gate_add_kernel, and the
// gate and add of the fused lookup).
//
// Per token, with a = stream 0, ra = (|a|^2/D + eps)^-1/2, rk likewise for k,
// z = ra rk <a, k> / sqrt(D), g = sigmoid(z), c = sum_s alpha_s dy_s:
//   d<loss>/dz = dz = <c, k> g (1 - g)
//   dk   = g c + dz (ra rk / sqrt(D) a - z rk^2 / D k)
//   dx_0 = dy_0 + dz (ra rk / sqrt(D) k - z ra^2 / D a),   dx_s = dy_s (s > 0)
//   dalpha_s = sum_t g <dy_s, k>
// (the derivative of ra is -ra^3 a / D, which is where the second terms come from).
//
// HBM-bound: 10D + 4D bytes in, 8D + 4D (2D for a bf16 dk) out per token, nothing
// read twice.  A token's k, stream 0 and four gradient streams stay in the
// registers of its threads (8 columns each: 16-byte accesses, neighbouring lanes
// adjacent) between the reduction of the seven sums (|a|^2, |k|^2, <a,k>, <dy_s,k>)
// and the stores.  Tokens wider than 256 take a block at a time (D/8 threads), two such
// blocks an SM at D = 4096, so that one's sums and stores run under the other's loads.
// (Bulk copies into a ring of shared-memory stages under the same arithmetic were
// slower everywhere: 1104 us against 1054 at 65,536 x 4096, 17.1 against 13.0 at 512 x
// 4096, 7.7 against 6.5 at 1024 x 1024.)  Narrower tokens take a power of two lanes of
// a warp (262,144 x 128: 141 us, 163 a block at a time; x 256: 278 and 285).  dalpha crosses tokens: each
// block adds its tokens in order and writes one partial; a second launch of one block adds
// the partials as a tree in a fixed order, so the result does not depend on timing.
// Measured: 65,536 x 4096 1054 us (26 D bytes a token: 6.6 TB/s), 512 x 4096 13 us
// (the load, sums and stores of two tokens, one after the other, and the second launch).
// A block of more than 512 threads would have an SM to itself and overlap nothing, so wider
// tokens take a pair of CTAs (a cluster), half of the columns each, whose sums meet through
// distributed shared memory: 32,768 x 8192 1291 us, a block a token 1531.
#include <atomic>

#include "launch.cuh"
#include "lookup_common.cuh"
#include "tensor_core.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr uint8_t kDead = 1, kBad = 2;

struct Cols {
  float k[8];
  uint4 a, dy[4];
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = bf16_lo(w[q]);
    f[2 * q + 1] = bf16_hi(w[q]);
  }
}

__device__ __forceinline__ void load_cols(Cols &c, const GateGradParams &p, int64_t t, int col) {
  const int64_t D = p.D;
  const float4 *kr = reinterpret_cast<const float4 *>(p.k + t * D + col);
  const float4 k0 = __ldcs(kr), k1 = __ldcs(kr + 1);
  c.a = __ldcs(reinterpret_cast<const uint4 *>(p.x + t * 4 * D + col));
#pragma unroll
  for (int s = 0; s < 4; ++s)
    c.dy[s] = __ldcs(reinterpret_cast<const uint4 *>(p.dy + (t * 4 + s) * D + col));
  c.k[0] = k0.x, c.k[1] = k0.y, c.k[2] = k0.z, c.k[3] = k0.w;
  c.k[4] = k1.x, c.k[5] = k1.y, c.k[6] = k1.z, c.k[7] = k1.w;
}

// This thread's part of the seven sums: |a|^2, |k|^2, <a,k>, <dy_s,k>.
__device__ __forceinline__ void partial_sums(const Cols &c, float (&r)[7]) {
  float f[8];
  unpack8(c.a, f);
#pragma unroll
  for (int i = 0; i < 7; ++i) r[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[0] = fmaf(f[i], f[i], r[0]);
    r[1] = fmaf(c.k[i], c.k[i], r[1]);
    r[2] = fmaf(f[i], c.k[i], r[2]);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    unpack8(c.dy[s], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[3 + s] = fmaf(f[i], c.k[i], r[3 + s]);
  }
}

struct Gate {
  float g, cross, wa, wk;  // dk = g c + cross a + wk k;  dx_0 = dy_0 + cross k + wa a
};

__device__ __forceinline__ Gate gate_of(const float (&r)[7], const float4 &alpha,
                                        const GateGradParams &p) {
  const float ra = rsqrtf(fmaf(r[0], p.inv_D, p.eps)), rk = rsqrtf(fmaf(r[1], p.inv_D, p.eps));
  const float u = ra * rk * p.inv_sqrt_D;
  const float z = r[2] * u;
  // sigmoid and its slope from exp(-|z|), which neither overflows nor cancels
  const float e = expf(-fabsf(z)), d = __fdividef(1.f, 1.f + e);
  const float dc = alpha.x * r[3] + alpha.y * r[4] + alpha.z * r[5] + alpha.w * r[6];
  const float dz = dc * (e * d * d);
  Gate o;
  o.g = z >= 0.f ? d : e * d;
  o.cross = dz * u;
  o.wa = -dz * z * ra * ra * p.inv_D;
  o.wk = -dz * z * rk * rk * p.inv_D;
  return o;
}

// The seven sums over a block.  A warp halves the number of values a lane holds at each of
// three exchanges, so 9 shuffles do for 35; lane 4i then has value i.  s_red: [7][warps].
__device__ __forceinline__ void warp_sums(const float (&r)[7], float *s_red, int warp, int warps, int lane) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < 7 ? r[i] : 0.f;
#pragma unroll
  for (int half = 4; half > 0; half >>= 1) {
    const bool up = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * half);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  if ((lane & 3) == 0 && lane < 28) s_red[(lane >> 2) * warps + warp] = v[0];
}

// .. and, behind a barrier, over its warps: a lane a warp, then a butterfly.  PAIR: over the
// warps of both CTAs, in the order of their ranks.
template <bool PAIR>
__device__ __forceinline__ void block_sums(float (&r)[7], const float *s_red, int warps, int lane) {
  const int rank = PAIR && lane >= warps;
  const uint32_t from = PAIR ? map_to_rank(smem_u32(s_red), rank) + (lane - rank * warps) * 4 : 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    float v = 0.f;
    if constexpr (PAIR) {
      if (lane < 2 * warps)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + i * warps * 4) : "memory");
    } else {
      if (lane < warps) v = s_red[i * warps + lane];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    r[i] = v;
  }
}

template <typename TK>
__device__ __forceinline__ void store_dk(TK *dk, const float (&v)[8]) {
  if constexpr (sizeof(TK) == 4) {
    __stcs(reinterpret_cast<float4 *>(dk), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(dk) + 1, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    __stcs(reinterpret_cast<uint4 *>(dk), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                      pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
  }
}

template <typename TK>
__device__ __forceinline__ void store_cols(const Cols &c, const Gate &o, const float4 &alpha,
                                           const GateGradParams &p, int64_t t, int col) {
  const int64_t D = p.D;
  float a[8], y[8], v[8];
  unpack8(c.a, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(o.cross, a[i], o.wk * c.k[i]);
  const float al[4] = {alpha.x, alpha.y, alpha.z, alpha.w};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    unpack8(c.dy[s], y);
    const float ga = o.g * al[s];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(ga, y[i], v[i]);
  }
  store_dk(static_cast<TK *>(p.dk) + t * D + col, v);
  unpack8(c.dy[0], y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] += fmaf(o.cross, c.k[i], o.wa * a[i]);
  uint16_t *dx = p.dx + t * 4 * D + col;
  __stcs(reinterpret_cast<uint4 *>(dx), make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                    pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])));
  if (p.dx != p.dy) {
#pragma unroll
    for (int s = 1; s < 4; ++s) __stcs(reinterpret_cast<uint4 *>(dx + s * D), c.dy[s]);
  }
}

// A token without a gate: dk = 0, and dy passed through when it is dead.
template <typename TK>
__device__ __forceinline__ void store_dead(const GateGradParams &p, uint8_t state, int64_t t,
                                           int col) {
  const int64_t D = p.D;
  const float zero[8] = {};
  store_dk(static_cast<TK *>(p.dk) + t * D + col, zero);
  if (state == kDead && p.dx != p.dy) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t o = (t * 4 + s) * D + col;
      __stcs(reinterpret_cast<uint4 *>(p.dx + o), __ldcs(reinterpret_cast<const uint4 *>(p.dy + o)));
    }
  }
}

// One token a block at a time, threads = D/8 rounded up to warps; PAIR: a token a pair of
// CTAs (a cluster), half of its columns each.
template <typename TK, bool PAIR>
__global__ void __launch_bounds__(512, 2) gate_grad_block_kernel(const __grid_constant__ GateGradParams p) {
  __shared__ float s_red[2][7 * 16];  // two tokens in turn: one barrier a token
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int width = PAIR ? p.D / 2 : p.D;
  const bool mine = tid * 8 < width;
  const int col = PAIR ? (int)cluster_rank() * width + tid * 8 : tid * 8;
  const int64_t first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
  const float4 alpha = make_float4(__ldg(p.alpha), __ldg(p.alpha + 1), __ldg(p.alpha + 2),
                                   __ldg(p.alpha + 3));
  float4 da = make_float4(0.f, 0.f, 0.f, 0.f);
  int buf = 0;
  for (int64_t t = first; t < p.T; t += step) {
    const uint8_t state = p.state ? p.state[t] : 0;  // the same in the whole block or pair
    if (state == kDead || state == kBad) {
      if (mine) store_dead<TK>(p, state, t, col);
      continue;
    }
    Cols c;
    float r[7] = {};
    if (mine) {
      load_cols(c, p, t, col);
      partial_sums(c, r);
    }
    warp_sums(r, s_red[buf], warp, warps, lane);
    if constexpr (PAIR)
      cluster_sync();
    else
      __syncthreads();
    block_sums<PAIR>(r, s_red[buf], warps, lane);
    buf ^= 1;
    const Gate o = gate_of(r, alpha, p);
    da.x = fmaf(o.g, r[3], da.x), da.y = fmaf(o.g, r[4], da.y);
    da.z = fmaf(o.g, r[5], da.z), da.w = fmaf(o.g, r[6], da.w);
    if (mine) store_cols<TK>(c, o, alpha, p, t, col);
  }
  if constexpr (PAIR) cluster_sync();  // no CTA leaves while the other may still read its sums
  if (tid == 0 && (!PAIR || cluster_rank() == 0)) p.partial[first] = da;
}

// Narrow tokens (D <= 256): p.group lanes a token, 256 / group tokens a block.
template <typename TK>
__global__ void __launch_bounds__(256) gate_grad_warp_kernel(const __grid_constant__ GateGradParams p) {
  __shared__ float4 s_da[128];
  dependency_wait();
  const int tid = threadIdx.x, G = p.group;
  const int in = tid & (G - 1), slot = tid / G, slots = 256 / G;
  const int col = in * 8;
  const bool mine = col < p.D;
  const float4 alpha = make_float4(__ldg(p.alpha), __ldg(p.alpha + 1), __ldg(p.alpha + 2),
                                   __ldg(p.alpha + 3));
  float4 da = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t t0 = (int64_t)blockIdx.x * slots; t0 < p.T; t0 += (int64_t)gridDim.x * slots) {
    const int64_t t = t0 + slot;
    const bool have = t < p.T;
    const uint8_t state = have && p.state ? p.state[t] : 0;
    const bool live = have && state != kDead && state != kBad;
    Cols c;
    float r[7] = {};
    if (live && mine) {
      load_cols(c, p, t, col);
      partial_sums(c, r);
    }
    for (int o = G >> 1; o > 0; o >>= 1)  // the group's lanes
#pragma unroll
      for (int i = 0; i < 7; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
    if (live) {
      const Gate o = gate_of(r, alpha, p);
      da.x = fmaf(o.g, r[3], da.x), da.y = fmaf(o.g, r[4], da.y);
      da.z = fmaf(o.g, r[5], da.z), da.w = fmaf(o.g, r[6], da.w);
      if (mine) store_cols<TK>(c, o, alpha, p, t, col);
    } else if (have && mine) {
      store_dead<TK>(p, state, t, col);
    }
  }
  if (in == 0) s_da[slot] = da;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < slots; ++i) {
      const float4 v = s_da[i];
      da.x += v.x, da.y += v.y, da.z += v.z, da.w += v.w;
    }
    p.partial[blockIdx.x] = da;
  }
}

__global__ void __launch_bounds__(256) dalpha_kernel(const float4 *__restrict__ partial, int n,
                                                     float *__restrict__ dalpha) {
  __shared__ float s[8][4];
  dependency_wait();
  float v[4] = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < n; i += 256) {
    const float4 q = partial[i];
    v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[threadIdx.x >> 5][i] = v[i];
  __syncthreads();
  if (threadIdx.x < 4) {
    float t = 0;
    for (int w = 0; w < 8; ++w) t += s[w][threadIdx.x];
    dalpha[threadIdx.x] = t;
  }
}

// Blocks that fit on the device at once, asked once per kernel, block size and device.
template <void (*kernel)(GateGradParams)>
cudaError_t resident_blocks(int threads, int &blocks) {
  static std::atomic<int> known[64][33];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int> &slot = known[dev & 63][threads / 32];
  blocks = slot.load(std::memory_order_relaxed);
  if (blocks) return cudaSuccess;
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0);
  if (e != cudaSuccess) return e;
  blocks = per * sms < kGateGradMaxBlocks ? per * sms : kGateGradMaxBlocks;
  slot.store(blocks, std::memory_order_relaxed);
  return cudaSuccess;
}

template <typename TK>
cudaError_t launch_typed(GateGradParams p, cudaStream_t stream) {
  int n = 0;
  p.inv_D = 1.f / (float)p.D;
  p.inv_sqrt_D = 1.f / sqrtf((float)p.D);
  if (p.T > 0) {
    const int chunks = p.D / 8;
    cudaError_t e;
    if (chunks <= 32) {
      p.group = 2;
      while (p.group < chunks) p.group *= 2;
      const int64_t need = (p.T + 256 / p.group - 1) / (256 / p.group);
      if ((e = resident_blocks<gate_grad_warp_kernel<TK>>(256, n)) != cudaSuccess) return e;
      n = (int)(need < n ? need : n);
      e = launch(gate_grad_warp_kernel<TK>, n, 256, 0, stream, 1, p);
    } else if (chunks <= 512) {
      const int threads = (chunks + 31) / 32 * 32;
      if ((e = resident_blocks<gate_grad_block_kernel<TK, false>>(threads, n)) != cudaSuccess) return e;
      n = (int)(p.T < n ? p.T : n);
      e = launch(gate_grad_block_kernel<TK, false>, n, threads, 0, stream, 1, p);
    } else {
      const int threads = (chunks / 2 + 31) / 32 * 32;
      if ((e = resident_blocks<gate_grad_block_kernel<TK, true>>(threads, n)) != cudaSuccess) return e;
      n = (int)(p.T < n / 2 ? p.T : n / 2);
      e = launch(gate_grad_block_kernel<TK, true>, 2 * (int64_t)n, threads, 0, stream, 2, p);
    }
    if (e != cudaSuccess) return e;
  }
  return launch(dalpha_kernel, 1, 256, 0, stream, 1, p.partial, n, p.dalpha);
}

}  // namespace

cudaError_t launch_gate_grad(const GateGradParams &p, int dk_dtype, cudaStream_t stream) {
  return dk_dtype == ENGRAM_DTYPE_F32 ? launch_typed<float>(p, stream)
                                      : launch_typed<uint16_t>(p, stream);
}

}  // namespace engram

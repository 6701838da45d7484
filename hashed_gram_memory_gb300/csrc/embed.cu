// embed.cu -- rows of one table looked up by id, scaled, and optionally summed
// over a token's ids.
//
// HBM-bound: a row is read (4 or 2 bytes a value) and written once; neighbouring lanes take
// neighbouring columns, 8 of them where rows are on 16-byte boundaries.
//   rows kernel (many rows of 2^i or 256 j columns): a warp takes 32 output rows, its
//     lanes first their ids and places, one each; then the rows go through the warp, four
//     loads in flight a lane, with two shuffles for what the flat kernel computes per
//     thread (1,572,864 rows of 256 bf16: 225 us, 94 % of the measured copy bandwidth);
//   columns kernel (rows wider than 32 that are not on 16-byte boundaries): the same with
//     fewer rows a warp and a column a lane;
//   flat kernel (few rows, other widths): a thread an output chunk (one row of 4096: 1.4 us);
//   pooled outputs (flat): a thread loops over the token's ids in order, four rows in
//     flight, in fp32 (65,536 x 24 ids of 256 bf16: 133 us, its bytes take 115 at the copy
//     bandwidth; 4096 x 6 of 256: 3.4 of 2.2; 20,000 x 6 of 475, a column a thread: 84 of 13).
#include "launch.cuh"
#include "lookup_common.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;

template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * sizeof(T) / 16;
  uint4 w[kWords];
};
template <>
struct Raw<float, 1> {
  float v;
};
template <>
struct Raw<uint16_t, 1> {
  uint16_t v;
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *src) {
  Raw<T, V> r;
  if constexpr (V == 1) {
    r.v = __ldg(src);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kWords; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void to_float(const Raw<T, V> &r, float (&f)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4)
      f[0] = r.v;
    else
      f[0] = bf16_lo(r.v);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kWords; ++i) {
      const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 4) {
          f[4 * i + q] = __uint_as_float(w[q]);
        } else {
          f[8 * i + 2 * q] = bf16_lo(w[q]);
          f[8 * i + 2 * q + 1] = bf16_hi(w[q]);
        }
      }
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_float(T *dst, const float (&f)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4)
      *dst = f[0];
    else
      *dst = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  } else if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4 *>(dst), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
  }
}

// Output rows times column chunks, numbered along the rows; a block takes
// kThreads * U consecutive ones.  `magic` is ceil(2^32 / chunks): a block's local
// numbers are below chunks + kThreads * U, where the multiplication is exact.
template <typename TI, typename TO, int V, int U, bool POOLED>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const __grid_constant__ EmbedParams p, int32_t chunks, uint32_t magic) {
  dependency_wait();
  const int64_t base = (int64_t)blockIdx.x * (kThreads * U);
  const int64_t row0 = base / chunks;
  const uint32_t rem0 = (uint32_t)(base - row0 * chunks);
  const int64_t n_rows = POOLED ? p.n_tokens : p.n_tokens * p.n_ids;
  const TI *table = static_cast<const TI *>(p.table);
  int64_t row[U];
  int col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t x = rem0 + u * kThreads + threadIdx.x;
    const uint32_t q = chunks == 1 ? x : __umulhi(x, magic);
    row[u] = row0 + q;
    col[u] = (int)(x - q * chunks) * V;
  }
  if constexpr (!POOLED) {
    int32_t id[U];
    int64_t at[U];
    Raw<TI, V> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      id[u] = ENGRAM_ROW_DEAD - 1;
      if (row[u] < n_rows) {
        const uint32_t r32 = (uint32_t)row[u];  // n_tokens * n_ids < 2^31
        const uint32_t t = fast_div(r32, p.by_ids), j = r32 - t * (uint32_t)p.n_ids;
        id[u] = __ldg(p.ids + t * p.ids_stride + j);
        at[u] = t * p.out_token_stride + j * p.out_id_stride;
        if (id[u] < ENGRAM_ROW_DEAD || id[u] >= p.rows) {
          if (col[u] == 0 && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
          id[u] = ENGRAM_ROW_DEAD - 1;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] >= 0) raw[u] = load_raw<TI, V>(table + id[u] * p.table_stride + col[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (id[u] < ENGRAM_ROW_DEAD) continue;
      float f[V] = {};
      if (id[u] >= 0) {
        to_float<TI, V>(raw[u], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= p.scale;
      }
      store_float<TO, V>(static_cast<TO *>(p.out) + at[u] + col[u], f);
    }
  } else {
    static_assert(U == 1);
    constexpr int kAhead = 4;
    if (row[0] >= n_rows) return;
    const int32_t *ids = p.ids + row[0] * p.ids_stride;
    float acc[V] = {};
    bool bad = false;
    for (int j0 = 0; j0 < p.n_ids; j0 += kAhead) {
      int32_t id[kAhead];
      Raw<TI, V> raw[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        id[a] = j0 + a < p.n_ids ? __ldg(ids + j0 + a) : ENGRAM_ROW_DEAD;
        if (id[a] < ENGRAM_ROW_DEAD || id[a] >= p.rows) {
          bad = true;
          id[a] = ENGRAM_ROW_DEAD;
        }
        if (id[a] >= 0) raw[a] = load_raw<TI, V>(table + id[a] * p.table_stride + col[0]);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (id[a] < 0) continue;
        float f[V];
        to_float<TI, V>(raw[a], f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += f[i];
      }
    }
    if (bad) {
      if (col[0] == 0 && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= p.scale;
    store_float<TO, V>(static_cast<TO *>(p.out) + row[0] * p.out_token_stride + col[0], acc);
  }
}

// A lane's output row: its id (under ENGRAM_ROW_DEAD when the row stays unwritten) and place.
__device__ __forceinline__ void lane_row(const EmbedParams &p, int64_t row, bool flags, int32_t &id, int64_t &at) {
  id = ENGRAM_ROW_DEAD - 1;
  at = 0;
  if (row >= p.n_tokens * p.n_ids) return;
  const uint32_t t = fast_div((uint32_t)row, p.by_ids), j = (uint32_t)row - t * (uint32_t)p.n_ids;
  id = __ldg(p.ids + t * p.ids_stride + j);
  at = t * p.out_token_stride + j * p.out_id_stride;
  if (id < ENGRAM_ROW_DEAD || id >= p.rows) {
    if (flags && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
    id = ENGRAM_ROW_DEAD - 1;
  }
}

// Output rows in batches of 32 a warp: G lanes a row (p.D = 8 G, or G = 32 and 256 columns
// a slab), U rows in flight a lane.
template <typename TI, typename TO, int U>
__global__ void __launch_bounds__(kThreads)
    embed_rows_kernel(const __grid_constant__ EmbedParams p, int32_t G, int32_t slabs) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t batch = unit / slabs;
  const int slab = (int)(unit - batch * slabs);
  const int64_t n_rows = p.n_tokens * p.n_ids, row = batch * 32 + lane;
  if (batch * 32 >= n_rows) return;
  int32_t id;
  int64_t at;
  lane_row(p, row, slab == 0, id, at);
  const int per = 32 / G, mine = lane / G;  // rows side by side in a warp
  const int col = (slab * 32 + (lane & (G - 1))) * 8;
  const TI *table = static_cast<const TI *>(p.table) + col;
  TO *out = static_cast<TO *>(p.out) + col;
  for (int i = 0; i < G; i += U) {
    Raw<TI, 8> raw[U];
    int32_t ids[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ids[u] = __shfl_sync(0xffffffffu, id, (i + u) * per + mine);
      if (ids[u] >= 0) raw[u] = load_raw<TI, 8>(table + ids[u] * p.table_stride);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t to = __shfl_sync(0xffffffffu, at, (i + u) * per + mine);
      if (ids[u] < ENGRAM_ROW_DEAD) continue;
      float f[8] = {};
      if (ids[u] >= 0) {
        to_float<TI, 8>(raw[u], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] *= p.scale;
      }
      store_float<TO, 8>(out + to, f);
    }
  }
}

// Rows that are not on 16-byte boundaries, `batch` of them a warp: a column a lane, 8 values in
// flight a lane -- 32 W columns of 8 / W rows at a time.
template <typename TI, typename TO, int W>
__global__ void __launch_bounds__(kThreads)
    embed_columns_kernel(const __grid_constant__ EmbedParams p, int32_t batch) {
  dependency_wait();
  constexpr int kRows = 8 / W;
  const int lane = threadIdx.x & 31;
  const int64_t first = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * batch;
  int32_t id = ENGRAM_ROW_DEAD - 1;
  int64_t at = 0;
  if (lane < batch) lane_row(p, first + lane, true, id, at);
  const TI *src = static_cast<const TI *>(p.table) + (id >= 0 ? id : 0) * p.table_stride;
  TO *dst = static_cast<TO *>(p.out) + at;
  for (int i = 0; i < batch; i += kRows) {
    int32_t ids[kRows];
    const TI *from[kRows];
    TO *to[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      ids[r] = __shfl_sync(0xffffffffu, id, i + r);
      from[r] = reinterpret_cast<const TI *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), i + r));
      to[r] = reinterpret_cast<TO *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), i + r));
    }
    for (int c0 = lane; c0 < p.D; c0 += 32 * W) {
      Raw<TI, 1> raw[kRows][W];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < W; ++c)
          if (ids[r] >= 0 && c0 + 32 * c < p.D) raw[r][c] = load_raw<TI, 1>(from[r] + c0 + 32 * c);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < W; ++c) {
          if (ids[r] < ENGRAM_ROW_DEAD || c0 + 32 * c >= p.D) continue;
          float f[1] = {0.f};
          if (ids[r] >= 0) {
            to_float<TI, 1>(raw[r][c], f);
            f[0] *= p.scale;
          }
          store_float<TO, 1>(to[r] + c0 + 32 * c, f);
        }
    }
  }
}

template <typename TI, typename TO, int V, bool POOLED>
cudaError_t launch_sized(const EmbedParams &p, cudaStream_t stream) {
  const int32_t chunks = (p.D + V - 1) / V;
  const uint32_t magic = (uint32_t)(((1ull << 32) + chunks - 1) / chunks);
  const int64_t n_rows = POOLED ? p.n_tokens : p.n_tokens * p.n_ids;
  const int64_t items = n_rows * chunks;
  if constexpr (!POOLED && V == 8) {
    // Warps of 32 rows where there are many for every SM's schedulers: bf16 rows of 256, 131,072
    // take 24.6 us so and 22.9 by the flat kernel, 262,144 41.6 and 43.0, 1,572,864 225 and 244;
    // rows of 64 columns, 98,304 5.2 and 4.5, 200,000 8.8 and 10.2, 1,600,000 42 and 59.
    const int G = chunks < 32 ? chunks : 32, slabs = chunks < 32 ? 1 : chunks / 32;
    const int64_t units = (n_rows + 31) / 32 * slabs;
    if (G >= 4 && (G & (G - 1)) == 0 && chunks % G == 0 && units >= kSms * (chunks < 32 ? 32 : 48)) {
      constexpr int U = sizeof(TI) == 4 ? 2 : 4;
      return launch(embed_rows_kernel<TI, TO, U>, (units + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0,
                    stream, 1, p, G, slabs);
    }
  }
  if constexpr (!POOLED && V == 1) {
    // Wider than a warp: a few rows a warp, so that the ids, places and divisions are worked out
    // once a row and not once a value: 197,000 x 475 bf16 69 us, a thread a value 260; 5000 x 475
    // 4.0 and 7.5; 500 x 475 1.7 and 1.9.  More warps than schedulers need beat more rows a warp
    // (32 warps an SM: 95 us).
    if (p.D > 32) {
      int32_t batch = p.D <= 64 ? 4 : p.D <= 128 ? 2 : 1;
      while (batch < 32 && n_rows >= kSms * 128 * 2 * batch) batch *= 2;
      const int64_t warps = (n_rows + batch - 1) / batch;
      return launch(p.D <= 64    ? embed_columns_kernel<TI, TO, 2>
                    : p.D <= 128 ? embed_columns_kernel<TI, TO, 4>
                                 : embed_columns_kernel<TI, TO, 8>,
                    (warps + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, stream, 1, p, batch);
    }
  }
  // Few items, or pooled ones (which loop over their ids): one a thread.
  if (POOLED || items <= kSms * 4 * kThreads) {
    return launch(embed_kernel<TI, TO, V, 1, POOLED>, (items + kThreads - 1) / kThreads, kThreads, 0, stream, 1,
                  p, chunks, magic);
  }
  if constexpr (!POOLED) {
    constexpr int U = 2;
    return launch(embed_kernel<TI, TO, V, U, POOLED>, (items + kThreads * U - 1) / (kThreads * U), kThreads, 0,
                  stream, 1, p, chunks, magic);
  }
  return cudaErrorInvalidValue;  // not reached
}

template <typename TI, typename TO>
cudaError_t launch_typed(const EmbedParams &p, bool pooled, cudaStream_t stream) {
  const bool vec = p.D % 8 == 0 && (p.table_stride * sizeof(TI)) % 16 == 0 &&
                   (p.out_token_stride * sizeof(TO)) % 16 == 0 &&
                   (pooled || (p.out_id_stride * sizeof(TO)) % 16 == 0) &&
                   ((uintptr_t)p.table | (uintptr_t)p.out) % 16 == 0;
  if (vec)
    return pooled ? launch_sized<TI, TO, 8, true>(p, stream) : launch_sized<TI, TO, 8, false>(p, stream);
  return pooled ? launch_sized<TI, TO, 1, true>(p, stream) : launch_sized<TI, TO, 1, false>(p, stream);
}

}  // namespace

cudaError_t launch_embed(const EmbedParams &args, int table_dtype, int out_dtype, bool pooled,
                         cudaStream_t stream) {
  EmbedParams p = args;
  p.by_ids = fast_div_of((uint32_t)p.n_ids);
  if (table_dtype == ENGRAM_DTYPE_F32)
    return out_dtype == ENGRAM_DTYPE_F32 ? launch_typed<float, float>(p, pooled, stream)
                                         : launch_typed<float, uint16_t>(p, pooled, stream);
  return out_dtype == ENGRAM_DTYPE_F32 ? launch_typed<uint16_t, float>(p, pooled, stream)
                                       : launch_typed<uint16_t, uint16_t>(p, pooled, stream);
}

}  // namespace engram

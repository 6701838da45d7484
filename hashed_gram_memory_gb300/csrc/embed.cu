// embed.cu -- rows of one table looked up by id, scaled, and optionally summed
// over a token's ids.
//
// HBM-bound: a row is read (4 or 2 bytes a value) and written once.  Each thread
// handles 8 columns of an output row (one column on the path for odd widths and
// alignments), four outputs at a time, their loads issued together so that a warp
// keeps 2 KB in flight; neighbouring lanes read neighbouring columns.  A pooled
// output loops over the token's ids in order, four rows in flight, in fp32.
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
        const uint32_t t = r32 / (uint32_t)p.n_ids, j = r32 - t * (uint32_t)p.n_ids;
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

template <typename TI, typename TO, int V, bool POOLED>
cudaError_t launch_sized(const EmbedParams &p, cudaStream_t stream) {
  const int32_t chunks = (p.D + V - 1) / V;
  const uint32_t magic = (uint32_t)(((1ull << 32) + chunks - 1) / chunks);
  const int64_t n_rows = POOLED ? p.n_tokens : p.n_tokens * p.n_ids;
  const int64_t items = n_rows * chunks;
  // Few items, or pooled ones (which loop over their ids): one a thread.
  if (POOLED || items <= 152 * 4 * kThreads) {
    return launch(embed_kernel<TI, TO, V, 1, POOLED>, (items + kThreads - 1) / kThreads, kThreads, 0, stream, 1,
                  p, chunks, magic);
  }
  if constexpr (!POOLED) {
    constexpr int U = 4;
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

cudaError_t launch_embed(const EmbedParams &p, int table_dtype, int out_dtype, bool pooled,
                         cudaStream_t stream) {
  if (table_dtype == ENGRAM_DTYPE_F32)
    return out_dtype == ENGRAM_DTYPE_F32 ? launch_typed<float, float>(p, pooled, stream)
                                         : launch_typed<float, uint16_t>(p, pooled, stream);
  return out_dtype == ENGRAM_DTYPE_F32 ? launch_typed<uint16_t, float>(p, pooled, stream)
                                       : launch_typed<uint16_t, uint16_t>(p, pooled, stream);
}

}  // namespace engram

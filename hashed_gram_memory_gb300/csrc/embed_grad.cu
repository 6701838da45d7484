// embed_grad.cu -- the gradient of an embedding lookup by sorted ids:
//   grad[v] (+)= scale * sum over positions i with ids[i] = v, in ascending i, of dy[i]
// as a dense [rows, D] gradient, or as the distinct ids and their rows.
//
// 1. Sort (id, position) pairs by id, stably: a radix sort, 8 bits a pass at most.  Up to
//    4096 ids run all passes in one block's shared memory; more take three launches a
//    pass (digit counts per tile of 4096, their prefix sums per digit, the scatter).  Dead
//    and bad ids get the key `rows`, which sorts behind every row.
// 2. Sum the runs of equal ids.  The sorted list is cut into chunks of equal length, a
//    group of lanes (8 columns a lane) walks a chunk with the rows of dy that come next
//    in flight, adds in fp32 and writes each run that lies inside its chunk; a run that
//    crosses a chunk's border leaves a partial sum there.  The chunks' equal length is what
//    keeps a token that makes up a tenth of the text from running on one SM.
// 3. Add the partial sums of each crossing run, in chunk order.
// Every sum has one order, so results do not depend on timing; there are no atomics on
// values.  A dense gradient's untouched rows are zeroed by further blocks of the second
// step's launch, which look each row up in the sorted list.
//
// HBM-bound: dy read once (scattered whole rows), each output row written once; the sort's
// lists stay in L2.
#include "launch.cuh"
#include "lookup_common.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr int kSortThreads = 512;
constexpr int kTile = 4096;             // pairs a tile of the sort
constexpr int kPer = kTile / kSortThreads;
constexpr int kSortWarps = kSortThreads / 32;

// x / d for x < 2^31: exact with m = ceil(2^(31 + l) / d), l = ceil(log2 d) (m < 2^32).
__device__ __forceinline__ uint32_t fast_div(uint32_t x, const FastDiv &f) {
  return (uint32_t)(((uint64_t)x * f.mul) >> f.shift);
}

// The sort key of position i: its id, or `rows` where it takes no part.
__device__ __forceinline__ uint32_t key_of(const EmbedGradParams &p, uint32_t i, bool &bad) {
  const uint32_t t = fast_div(i, p.by_ids), j = i - t * (uint32_t)p.n_ids;
  const int32_t id = __ldg(p.ids + t * p.ids_stride + j);
  if (id >= 0 && id < p.rows) return (uint32_t)id;
  bad |= id != ENGRAM_ROW_DEAD;
  return (uint32_t)p.rows;
}

// Stable ranks of a tile's pairs by one digit.  Warp w holds pairs w*32*kPer .. in order,
// pair (round r, lane l) at w*32*kPer + 32 r + l; slots at or past n are left out.  On
// return place[r] is the pair's position among the tile's pairs sorted by digit, and
// s_start[d] the first position of digit d.
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[kPer], int n, int shift, uint32_t mask,
                                          uint32_t (*s_cnt)[256], uint32_t *s_start,
                                          uint32_t (&place)[kPer]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kSortWarps * 256; i += kSortThreads) (&s_cnt[0][0])[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const bool have = warp * 32 * kPer + 32 * r + lane < n;
    const uint32_t d = have ? (key[r] >> shift) & mask : 256;
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const uint32_t before = __popc(same & ((1u << lane) - 1));
    if (have) {
      place[r] = s_cnt[warp][d] + before;
      __syncwarp(same);
      if (before == 0) s_cnt[warp][d] += __popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  // Exclusive prefix over the warps of each digit, then over the digits (256 threads).
  uint32_t total = 0, sum = 0;
  if (tid < 256) {
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = s_cnt[w][tid];
      s_cnt[w][tid] = total;
      total += c;
    }
    sum = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_start[warp] = sum;
  }
  __syncthreads();
  uint32_t base = 0;
  if (tid < 256)
    for (int w = 0; w < warp; ++w) base += s_start[w];
  __syncthreads();
  if (tid < 256) s_start[tid] = base + sum - total;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPer; ++r)
    if (warp * 32 * kPer + 32 * r + lane < n) {
      const uint32_t d = (key[r] >> shift) & mask;
      place[r] += s_cnt[warp][d] + s_start[d];
    }
}

// All passes of at most kTile pairs, then (for the sparse form) the number of runs that
// start before each chunk.
__global__ void __launch_bounds__(kSortThreads)
    sort_small_kernel(const __grid_constant__ EmbedGradParams p) {
  __shared__ uint32_t s_key[kTile];
  __shared__ uint16_t s_pos[kTile];
  __shared__ uint32_t s_cnt[kSortWarps][256];
  __shared__ uint32_t s_start[256];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)p.n;
  uint32_t key[kPer], pos[kPer], place[kPer];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    pos[r] = warp * 32 * kPer + 32 * r + lane;
    if (pos[r] < (uint32_t)n) key[r] = key_of(p, pos[r], bad);
  }
  if (bad && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
  for (int pass = 0; pass < p.passes; ++pass) {
    rank_tile(key, n, pass * p.digit_bits, (1u << p.digit_bits) - 1, s_cnt, s_start, place);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      if (warp * 32 * kPer + 32 * r + lane < n) {
        s_key[place[r]] = key[r];
        s_pos[place[r]] = (uint16_t)pos[r];
      }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int i = warp * 32 * kPer + 32 * r + lane;
      if (i < n) {
        key[r] = s_key[i];
        pos[r] = s_pos[i];
      }
    }
  }
  for (int i = tid; i < n; i += kSortThreads) {
    p.keys[i] = s_key[i];
    p.pos[i] = s_pos[i];
  }
  if (!p.run_base) return;
  // Runs starting in each of this thread's entries, then prefix sums over the entries.
  uint32_t mine = 0;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int i = tid * kPer + r;
    mine += i < n && s_key[i] < (uint32_t)p.rows && (i == 0 || s_key[i - 1] != s_key[i]);
  }
  uint32_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s_start[warp] = sum;
  __syncthreads();
  uint32_t at = sum - mine;
  for (int w = 0; w < warp; ++w) at += s_start[w];
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int i = tid * kPer + r;
    if (i < n && i % p.chunk == 0) p.run_base[i / p.chunk] = at;
    at += i < n && s_key[i] < (uint32_t)p.rows && (i == 0 || s_key[i - 1] != s_key[i]);
  }
  if (tid == kSortThreads - 1) {
    p.run_base[p.chunks] = at;
    *p.count_out = (int32_t)at;
  }
}

// ---- one pass of the sort of many pairs -----------------------------------------------

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    count_digits_kernel(const __grid_constant__ EmbedGradParams p, const uint32_t *__restrict__ keys,
                        int shift) {
  __shared__ uint32_t s_cnt[256];
  dependency_wait();
  const int tid = threadIdx.x;
  const uint32_t mask = (1u << p.digit_bits) - 1;
  if (tid < 256) s_cnt[tid] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int64_t i = base + r * kSortThreads + tid;
    if (i < p.n) {
      const uint32_t k = FIRST ? key_of(p, (uint32_t)i, bad) : __ldg(keys + i);
      atomicAdd(&s_cnt[(k >> shift) & mask], 1u);
    }
  }
  if (FIRST && bad && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
  __syncthreads();
  if (tid <= (int)mask) p.counts[(int64_t)tid * p.tiles + blockIdx.x] = s_cnt[tid];
}

// Block d: the counts of digit d become their exclusive prefix sums over the tiles; the
// digit's total goes behind the array.
__global__ void __launch_bounds__(256) scan_digits_kernel(uint32_t *counts, int64_t tiles,
                                                          uint32_t *totals) {
  __shared__ uint32_t s_sum[8];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t *c = counts + blockIdx.x * tiles;
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < tiles; i0 += 256) {
    const uint32_t v = i0 + tid < tiles ? c[i0 + tid] : 0;
    uint32_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    uint32_t before = carry, all = carry;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (i0 + tid < tiles) c[i0 + tid] = before + sum - v;
    carry = all;
    __syncthreads();
  }
  if (tid == 0) totals[blockIdx.x] = carry;
}

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
    scatter_kernel(const __grid_constant__ EmbedGradParams p, const uint32_t *__restrict__ keys,
                   const uint32_t *__restrict__ poss, uint32_t *__restrict__ keys_out,
                   uint32_t *__restrict__ pos_out, int shift) {
  __shared__ uint32_t s_key[kTile];
  __shared__ uint16_t s_from[kTile];
  __shared__ uint32_t s_cnt[kSortWarps][256];
  __shared__ uint32_t s_start[256];
  __shared__ uint32_t s_sum[8];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mask = (1u << p.digit_bits) - 1;
  const int64_t base = (int64_t)blockIdx.x * kTile;
  const int n = (int)(p.n - base < kTile ? p.n - base : kTile);
  uint32_t key[kPer], place[kPer];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int i = warp * 32 * kPer + 32 * r + lane;
    if (i < n) key[r] = FIRST ? key_of(p, (uint32_t)(base + i), bad) : __ldg(keys + base + i);
  }
  rank_tile(key, n, shift, mask, s_cnt, s_start, place);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int i = warp * 32 * kPer + 32 * r + lane;
    if (i < n) {
      s_key[place[r]] = key[r];
      s_from[place[r]] = (uint16_t)i;
    }
  }
  // Where each digit of this tile goes: the digits' totals before it, this digit in the
  // tiles before this one, less its first position in the tile.
  uint32_t *s_to = &s_cnt[0][0];
  __syncthreads();
  uint32_t t = 0, sum = 0;
  if (tid < 256) {
    t = tid <= (int)mask ? __ldg(p.totals + tid) : 0;
    sum = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_sum[warp] = sum;
  }
  __syncthreads();
  if (tid <= (int)mask) {
    uint32_t b = sum - t;
    for (int w = 0; w < warp; ++w) b += s_sum[w];
    s_to[tid] = b + __ldg(p.counts + (int64_t)tid * p.tiles + blockIdx.x) - s_start[tid];
  }
  __syncthreads();
  for (int i = tid; i < n; i += kSortThreads) {
    const uint32_t k = s_key[i];
    const uint32_t to = s_to[(k >> shift) & mask] + i;
    const uint32_t from = (uint32_t)base + s_from[i];
    keys_out[to] = k;
    pos_out[to] = FIRST ? from : __ldg(poss + from);
  }
}

// Runs that start in each chunk, a warp a chunk.
__global__ void __launch_bounds__(256) count_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  dependency_wait();
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (c >= p.chunks) return;
  const int64_t e0 = c * p.chunk, e1 = min(e0 + p.chunk, p.n);
  uint32_t mine = 0;
  for (int64_t e = e0 + lane; e < e1; e += 32) {
    const uint32_t k = __ldg(p.keys + e);
    mine += k < (uint32_t)p.rows && (e == 0 || __ldg(p.keys + e - 1) != k);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) p.run_base[c] = mine;
}

// run_base becomes its exclusive prefix sums; the number of runs goes behind it.
__global__ void __launch_bounds__(1024) scan_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  __shared__ uint32_t s_sum[32];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < p.chunks; i0 += 1024 * 8) {
    uint32_t v[8], mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = i0 + tid * 8 + i;
      v[i] = c < p.chunks ? p.run_base[c] : 0;
      mine += v[i];
    }
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    uint32_t at = carry + sum - mine, all = carry;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += s_sum[w];
      all += s_sum[w];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = i0 + tid * 8 + i;
      if (c < p.chunks) p.run_base[c] = at;
      at += v[i];
    }
    carry = all;
    __syncthreads();
  }
  if (tid == 0) {
    p.run_base[p.chunks] = carry;
    *p.count_out = (int32_t)carry;
  }
}

// ---- sums of runs ------------------------------------------------------------------------

template <typename T, int V>
struct Slice {  // V values of a row, as loaded
  uint4 w[V * sizeof(T) / 16];
  __device__ __forceinline__ void load(const T *src) {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
  }
  __device__ __forceinline__ void add_to(float (&acc)[V]) const {
#pragma unroll
    for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 4) {
          acc[4 * i + q] += __uint_as_float(u[q]);
        } else {
          acc[8 * i + 2 * q] += bf16_lo(u[q]);
          acc[8 * i + 2 * q + 1] += bf16_hi(u[q]);
        }
      }
    }
  }
};
template <typename T>
struct Slice<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T *src) { w = __ldg(src); }
  __device__ __forceinline__ void add_to(float (&acc)[1]) const {
    if constexpr (sizeof(T) == 4)
      acc[0] += w;
    else
      acc[0] += bf16_lo(w);
  }
};

// dst = scale * acc, or dst += scale * acc.
template <typename T, int V>
__device__ __forceinline__ void write_row(T *dst, const float (&acc)[V], float scale, bool accumulate) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = acc[i] * scale;
  if (accumulate) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4)
        f[i] += dst[i];
      else
        f[i] += bf16_lo(dst[i]);
    }
  }
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

template <int V>
__device__ __forceinline__ void write_partial(float *dst, const float (&acc)[V]) {
  if constexpr (V == 1) {
    *dst = acc[0];
  } else {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
}

constexpr uint32_t kNoKey = 0xFFFFFFFFu;
constexpr int kSumThreads = 128;

// A group's place: the chunk and the columns it works on.
struct Item {
  int64_t chunk;
  int slab, col, in;
};
__device__ __forceinline__ Item item_of(const EmbedGradParams &p, int64_t group, int in, int vec) {
  Item it;
  it.chunk = group / p.slabs;
  it.slab = (int)(group - it.chunk * p.slabs);
  it.in = in;
  it.col = (it.slab * p.group + in) * vec;
  return it;
}

template <typename TY, typename TG, int V, int U>
__device__ __forceinline__ void sum_chunk(const EmbedGradParams &p, const Item &it) {
  const int64_t e0 = it.chunk * p.chunk, e1 = min(e0 + p.chunk, p.n);
  const uint32_t rows = (uint32_t)p.rows;
  const bool mine = it.col < p.D;
  const bool lead = it.slab == 0 && it.in == 0;
  int64_t run = 0;
  if (p.run_base) {
    run = __ldg(p.run_base + it.chunk);
    if (it.slab == 0) {  // ids beyond the distinct ones
      const int64_t count = __ldg(p.run_base + p.chunks);
      for (int64_t e = e0 + it.in; e < e1; e += p.group)
        if (e >= count) p.row_ids_out[e] = ENGRAM_ROW_DEAD;
    }
  }
  uint32_t cur = __ldg(p.keys + e0);
  if (cur >= rows) return;
  bool open = e0 > 0 && __ldg(p.keys + e0 - 1) == cur;  // the run began in an earlier chunk
  if (open) --run;
  const TY *dy = static_cast<const TY *>(p.dy) + it.col;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const auto flush = [&](bool more) {
    if (open || more) {
      if (mine) write_partial<V>(p.partial + (it.chunk * 2 + (open ? 0 : 1)) * p.partial_stride + it.col, acc);
    } else {
      const int64_t row = p.run_base ? run : cur;
      if (mine)
        write_row<TG, V>(static_cast<TG *>(p.grad) + row * p.grad_stride + it.col, acc, p.scale, p.accumulate);
      if (p.run_base && lead) p.row_ids_out[run] = (int32_t)cur;
    }
  };
  for (int64_t e = e0; e < e1; e += U) {
    uint32_t key[U];
    Slice<TY, V> s[U];
#pragma unroll
    for (int u = 0; u < U; u += 4) {
      const uint4 k4 = __ldg(reinterpret_cast<const uint4 *>(p.keys + e + u));
      const uint4 p4 = __ldg(reinterpret_cast<const uint4 *>(p.pos + e + u));
      const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w}, pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        key[u + q] = e + u + q < e1 ? kk[q] : kNoKey;
        if (mine && key[u + q] < rows) {
          int64_t at = (int64_t)pp[q] * p.dy_id_stride;
          if (!p.dy_linear) {
            const uint32_t t = fast_div(pp[q], p.by_ids);
            at = t * p.dy_token_stride + (int64_t)(pp[q] - t * (uint32_t)p.n_ids) * p.dy_id_stride;
          }
          s[u + q].load(dy + at);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (key[u] == kNoKey) break;
      if (key[u] != cur) {
        flush(false);
        cur = key[u];
        if (cur >= rows) return;  // nothing but left-out positions follow
        open = false;
        ++run;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
      }
      if (mine) s[u].add_to(acc);
    }
  }
  flush(e1 < p.n && __ldg(p.keys + e1) == cur);
}

// 32 rows of a dense gradient: those that no id names are zeroed.
template <typename TG, int V>
__device__ __forceinline__ void zero_rows(const EmbedGradParams &p, int64_t r0) {
  const int lane = threadIdx.x & 31;
  const int64_t row = r0 + lane;
  bool zero = false;
  if (row < p.rows) {
    int64_t lo = 0, hi = p.n;  // the first key >= row
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (__ldg(p.keys + mid) < (uint32_t)row)
        lo = mid + 1;
      else
        hi = mid;
    }
    zero = lo >= p.n || __ldg(p.keys + lo) != (uint32_t)row;
  }
  uint32_t todo = __ballot_sync(0xffffffffu, zero);
  while (todo) {
    const int r = __ffs(todo) - 1;
    todo &= todo - 1;
    TG *dst = static_cast<TG *>(p.grad) + (r0 + r) * p.grad_stride;
    if constexpr (V == 1) {
      for (int c = lane; c < p.D; c += 32) dst[c] = TG(0);
    } else {
      for (int c = lane * (16 / (int)sizeof(TG)); c < p.D; c += 32 * (16 / (int)sizeof(TG)))
        __stcs(reinterpret_cast<uint4 *>(dst + c), make_uint4(0, 0, 0, 0));
    }
  }
}

template <typename TY, typename TG, int V, int U>
__global__ void __launch_bounds__(kSumThreads) sum_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  dependency_wait();
  if ((int64_t)blockIdx.x >= p.sum_blocks) {  // the zeroing blocks
    const int64_t w = (blockIdx.x - p.sum_blocks) * (kSumThreads / 32) + (threadIdx.x >> 5);
    if (w * 32 < p.rows) zero_rows<TG, V>(p, w * 32);
    return;
  }
  const int64_t group = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) / p.group;
  const Item it = item_of(p, group, threadIdx.x & (p.group - 1), V);
  if (it.chunk < p.chunks) sum_chunk<TY, TG, V, U>(p, it);
}

// ---- runs that cross chunks ----------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kAlone = 16;  // parts a group adds by itself

template <typename TG, int V>
__global__ void __launch_bounds__(kJoinThreads) join_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  extern __shared__ float s_part[];  // [groups a block][lanes a group * V]
  __shared__ int64_t s_parts[kJoinThreads];
  dependency_wait();
  const int G = p.group, groups = kJoinThreads / G;
  const int slot = threadIdx.x / G, in = threadIdx.x & (G - 1);
  const Item it = item_of(p, (int64_t)blockIdx.x * groups + slot, in, V);
  // The partial sums of the run that starts in this chunk and goes on after it.
  int64_t parts = 0;
  uint32_t key = kNoKey;
  if (it.chunk + 1 < p.chunks) {
    const int64_t e0 = it.chunk * p.chunk, e1 = e0 + p.chunk;
    key = __ldg(p.keys + e1 - 1);
    if (key < (uint32_t)p.rows && __ldg(p.keys + e1) == key &&
        !(e0 > 0 && __ldg(p.keys + e0 - 1) == key)) {
      int64_t lo = it.chunk + 1, hi = p.chunks;  // the first chunk that starts with another key
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(p.keys + mid * p.chunk) == key)
          lo = mid + 1;
        else
          hi = mid;
      }
      parts = lo - it.chunk;
    }
  }
  const auto part = [&](int64_t chunk, int64_t i, int col) {
    return p.partial + ((chunk + i) * 2 + (i == 0 ? 1 : 0)) * p.partial_stride + col;
  };
  const auto finish = [&](int64_t chunk, uint32_t k, int slab, int col, float (&acc)[V]) {
    const int64_t row = p.run_base ? (int64_t)__ldg(p.run_base + chunk + 1) - 1 : k;
    if (col < p.D) write_row<TG, V>(static_cast<TG *>(p.grad) + row * p.grad_stride + col, acc, p.scale, p.accumulate);
    if (p.run_base && slab == 0 && in == 0) p.row_ids_out[row] = (int32_t)k;
  };
  if (parts > 0 && parts <= kAlone) {
    float acc[V] = {};
    if (it.col < p.D)
      for (int64_t i = 0; i < parts; ++i) {
        Slice<float, V> s;
        s.load(part(it.chunk, i, it.col));
        s.add_to(acc);
      }
    finish(it.chunk, key, it.slab, it.col, acc);
  }
  if (in == 0) s_parts[slot] = parts;
  __syncthreads();
  // Longer runs take the whole block: each group adds every groups-th part, then the
  // first one adds the groups' sums in order.
  for (int o = 0; o < groups; ++o) {
    const int64_t n = s_parts[o];  // block-uniform
    if (n <= kAlone) continue;
    const Item other = item_of(p, (int64_t)blockIdx.x * groups + o, in, V);
    float acc[V] = {};
    if (other.col < p.D) {
#pragma unroll 4
      for (int64_t i = slot; i < n; i += groups) {
        Slice<float, V> s;
        s.load(part(other.chunk, i, other.col));
        s.add_to(acc);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s_part[(slot * G + in) * V + i] = acc[i];
    __syncthreads();
    if (slot == 0) {
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += s_part[(g * G + in) * V + i];
      finish(other.chunk, __ldg(p.keys + (other.chunk + 1) * p.chunk), other.slab, other.col, acc);
    }
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------------------

FastDiv fast_div_of(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  FastDiv f;
  f.shift = 31 + l;
  f.mul = (uint32_t)(((1ull << f.shift) + d - 1) / d);
  return f;
}

size_t round16(size_t x) { return (x + 15) / 16 * 16; }

// How the sums are cut: lanes a group, column slabs, chunk length.
struct Cut {
  int vec, group, slabs, chunk;
  int64_t chunks, stride;  // stride: columns of a partial sum's row
};
Cut cut_of(int64_t n, int D, bool vec) {
  Cut c;
  c.vec = vec ? 8 : 1;
  const int cols = (D + c.vec - 1) / c.vec;
  c.group = 1;
  while (c.group < 32 && c.group < cols) c.group *= 2;
  c.slabs = (cols + c.group - 1) / c.group;
  // Chunks long enough that partial sums are a small part of the traffic, short enough
  // that there are several warps for every SM's schedulers.
  c.chunk = 256;
  const int64_t warps = 152 * 48;
  while (c.chunk > 16 && (n + c.chunk - 1) / c.chunk * c.slabs * c.group / 32 < warps) c.chunk /= 2;
  // Short lists: shorter chunks still, while their partial sums stay under 2 MB.
  while (c.chunk > 4 && (n + c.chunk - 1) / c.chunk * c.slabs * c.group / 32 < warps / 8 &&
         (n / (c.chunk / 2) + 1) * 2 * (D + 8) * 4 <= (2 << 20))
    c.chunk /= 2;
  c.chunks = (n + c.chunk - 1) / c.chunk;
  c.stride = (D + 7) / 8 * 8;
  return c;
}

struct Layout {
  size_t keys[2], pos[2], counts, totals, run_base, partial, total;
};
Layout layout_of(int64_t n, int D, const Cut &c) {
  Layout l;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round16(bytes);
    return here;
  };
  const size_t list = (size_t)n * 4 + 64;  // read a few entries past the end (ignored)
  for (int i = 0; i < 2; ++i) {
    l.keys[i] = take(list);
    l.pos[i] = take(list);
  }
  l.counts = take((size_t)((n + kTile - 1) / kTile) * 256 * 4);
  l.totals = take(256 * 4);
  l.run_base = take((size_t)(c.chunks + 1) * 4);
  l.partial = take((size_t)c.chunks * 2 * c.stride * 4);
  l.total = at;
  return l;
}

template <typename TY, typename TG, int V>
cudaError_t launch_sums(EmbedGradParams p, cudaStream_t stream) {
  constexpr int U = V == 1 ? 8 : (sizeof(TY) == 4 ? 4 : 8);
  const int64_t groups = p.chunks * p.slabs;
  p.sum_blocks = (groups * p.group + kSumThreads - 1) / kSumThreads;
  const int64_t zero_blocks =
      p.run_base || p.accumulate ? 0 : (p.rows + kSumThreads - 1) / kSumThreads;  // a row a lane
  if (p.sum_blocks + zero_blocks > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (p.sum_blocks + zero_blocks > 0)
    e = launch(sum_runs_kernel<TY, TG, V, U>, p.sum_blocks + zero_blocks, kSumThreads, 0, stream, 1, p);
  if (e != cudaSuccess || p.chunks < 2) return e;
  const int per = kJoinThreads / p.group;
  return launch(join_runs_kernel<TG, V>, (groups + per - 1) / per, kJoinThreads,
                kJoinThreads * V * sizeof(float), stream, 1, p);
}

template <typename TY, typename TG>
cudaError_t launch_typed(const EmbedGradParams &p, bool vec, cudaStream_t stream) {
  return vec ? launch_sums<TY, TG, 8>(p, stream) : launch_sums<TY, TG, 1>(p, stream);
}

}  // namespace

size_t embed_grad_workspace_bytes(int64_t n, int32_t D) {
  // The larger of the two ways to cut (which one is used goes by alignment).
  const Cut a = cut_of(n, D, true), b = cut_of(n, D, false);
  const size_t x = layout_of(n, D, a).total, y = layout_of(n, D, b).total;
  return x > y ? x : y;
}

cudaError_t launch_embed_grad(EmbedGradParams p, int dy_dtype, int grad_dtype, void *workspace,
                              bool sparse, cudaStream_t stream) {
  const bool vec =
      p.D % 8 == 0 && ((uintptr_t)p.dy | (uintptr_t)p.grad) % 16 == 0 &&
      (p.dy_token_stride * dtype_bytes(dy_dtype)) % 16 == 0 &&
      (p.dy_id_stride * dtype_bytes(dy_dtype)) % 16 == 0 && (p.grad_stride * dtype_bytes(grad_dtype)) % 16 == 0;
  const Cut c = cut_of(p.n, p.D, vec);
  const Layout l = layout_of(p.n, p.D, c);
  char *w = static_cast<char *>(workspace);
  p.by_ids = fast_div_of((uint32_t)p.n_ids);
  p.dy_linear = p.dy_token_stride == p.n_ids * p.dy_id_stride;
  p.tiles = (p.n + kTile - 1) / kTile;
  p.counts = reinterpret_cast<uint32_t *>(w + l.counts);
  p.totals = reinterpret_cast<uint32_t *>(w + l.totals);
  p.run_base = sparse ? reinterpret_cast<uint32_t *>(w + l.run_base) : nullptr;
  p.partial = reinterpret_cast<float *>(w + l.partial);
  p.partial_stride = c.stride;
  p.group = c.group;
  p.slabs = c.slabs;
  p.chunk = c.chunk;
  p.chunks = c.chunks;
  int bits = 1;
  while (bits < 32 && ((uint64_t)p.rows >> bits) != 0) ++bits;  // keys are 0 .. rows
  p.passes = (bits + 7) / 8;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(w + l.keys[0]), reinterpret_cast<uint32_t *>(w + l.keys[1])};
  uint32_t *pos[2] = {reinterpret_cast<uint32_t *>(w + l.pos[0]), reinterpret_cast<uint32_t *>(w + l.pos[1])};
  cudaError_t e = cudaSuccess;
  p.keys = keys[0];
  p.pos = pos[0];
  if (p.n == 0) {
    if (sparse) return cudaMemsetAsync(p.count_out, 0, 4, stream);
  } else if (p.n <= kTile) {
    if ((e = launch(sort_small_kernel, 1, kSortThreads, 0, stream, 1, p)) != cudaSuccess) return e;
  } else {
    for (int pass = 0; pass < p.passes && e == cudaSuccess; ++pass) {
      const int shift = pass * p.digit_bits, in = pass & 1 ^ 1, out = pass & 1;
      e = launch(pass == 0 ? count_digits_kernel<true> : count_digits_kernel<false>, p.tiles, kSortThreads, 0,
                 stream, 1, p, keys[in], shift);
      if (e == cudaSuccess)
        e = launch(scan_digits_kernel, 1 << p.digit_bits, 256, 0, stream, 1, p.counts, p.tiles, p.totals);
      if (e == cudaSuccess)
        e = launch(pass == 0 ? scatter_kernel<true> : scatter_kernel<false>, p.tiles, kSortThreads, 0, stream, 1,
                   p, keys[in], pos[in], keys[out], pos[out], shift);
    }
    if (e != cudaSuccess) return e;
    p.keys = keys[(p.passes - 1) & 1];
    p.pos = pos[(p.passes - 1) & 1];
    if (sparse) {
      e = launch(count_runs_kernel, (p.chunks + 7) / 8, 256, 0, stream, 1, p);
      if (e == cudaSuccess) e = launch(scan_runs_kernel, 1, 1024, 0, stream, 1, p);
      if (e != cudaSuccess) return e;
    }
  }
  if (dy_dtype == ENGRAM_DTYPE_F32)
    return grad_dtype == ENGRAM_DTYPE_F32 ? launch_typed<float, float>(p, vec, stream)
                                          : launch_typed<float, uint16_t>(p, vec, stream);
  return grad_dtype == ENGRAM_DTYPE_F32 ? launch_typed<uint16_t, float>(p, vec, stream)
                                        : launch_typed<uint16_t, uint16_t>(p, vec, stream);
}

}  // namespace engram

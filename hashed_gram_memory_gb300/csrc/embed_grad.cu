// embed_grad.cu -- the gradient of an embedding lookup by sorted ids:
//   grad[v] (+)= scale * sum over positions i with ids[i] = v of dy[i]
// as a dense [rows, D] gradient, or as the distinct ids and their rows.  The order of a row's
// sum is fixed by the ids: ascending i, in parts where the id is frequent (2 and 3).
//
// 1. Sort (id, position) pairs by id, stably.  Up to 6144 ids: each id's place is the
//    number of ids before it in that order, counted by comparing it with all of them in
//    shared memory -- n^2 comparisons, but one launch over all SMs.  More: a radix sort, 10
//    bits a pass at most, three launches a pass (digit counts per tile, their prefix sums
//    per digit, the scatter).  Dead and bad ids get the key `rows`, which sorts behind
//    every row.
// 2. Sum the runs of equal ids.  The sorted list is cut into chunks of equal length; a
//    group of lanes (8 columns a lane) walks a chunk with the rows of dy that come next
//    in flight, adds in fp32 and writes each run that starts in its chunk, reading on into
//    the next chunk where the run ends there.  A run that goes on beyond the next chunk
//    leaves a partial sum for every chunk that it touches, and goes on a list: the chunks'
//    equal length is what keeps a token that makes up a tenth of the text from running on
//    one SM.
// 3. Add the partial sums of each listed run: a block's groups every groups-th one, ascending,
//    then the groups as a tree.
// Every sum has one order, so results do not depend on timing; there are no atomics on
// values.  A dense gradient's untouched rows are zeroed by further blocks of the second
// step's launch, spread evenly among the others, which look each row up in the sorted list.
//
// HBM-bound: dy read once (scattered whole rows), each output row written once; the sort's
// lists stay in L2.  Measured: 1,572,864 pairs of 256 bf16 columns into 1.30 M distinct rows
// 448 us, of which the sums 340 (2.1 GB of random 512-byte and 1 KB rows: 6.2 TB/s) and the
// sort, three passes of 10 bits, about 95; 16,384 x 4096 into a dense 129,280-row gradient
// 371 us (2.25 GB moved: 6.1 TB/s); 1536 pairs of 256 into 4096 rows 9.4 us (three launches,
// each waiting for the one before it).  Between them launches that are short and wait for one
// another take most of the time: distinct rows of 256 columns, 6144 pairs 22 us (their bytes
// take 1.4 at the copy bandwidth), 16,384 29 (3.6), 65,536 45 (15), 200,000 80 (43), 600,000
// 179 (111).
#include "bulk_copy.cuh"
#include "launch.cuh"
#include "lookup_common.cuh"
#include "train_internal.cuh"

namespace engram {
namespace {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kDigits = 1024;      // most digits of a pass: two a thread
// Most pairs sorted by counting: 4096 take 15.9 us in all so and 23.7 by digits, 6144 22.5 and
// 24.6, 8192 29.8 and 27.9.
constexpr int kCountSort = 6144;
constexpr uint32_t kNoKey = 0xFFFFFFFFu;
constexpr int kRunGroup = 16;      // chunks whose runs are counted together

// Pairs a thread sorts of a tile: few where there are few tiles, so that they fill the SMs
// (16,384 pairs take 31.6 us in all with two and 44.0 with eight, 600,000 179 and 186, 1,572,864
// 359 and 335).
constexpr int kPerLarge = 8, kPerSmall = 2;
constexpr int64_t kLargeTiles = kSms * kSortThreads * kPerLarge;  // from here on

// The sum of v over the threads before this one, of a block of kSortThreads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t *s_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane == 31) s_sum[warp] = sum;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
  return before + sum - v;
}

// The sort key of position i: its id, or `rows` where it takes no part.
__device__ __forceinline__ uint32_t key_of(const EmbedGradParams &p, uint32_t i, bool &bad) {
  const uint32_t t = fast_div(i, p.by_ids), j = i - t * (uint32_t)p.n_ids;
  const int32_t id = __ldg(p.ids + t * p.ids_stride + j);
  if (id >= 0 && id < p.rows) return (uint32_t)id;
  bad |= id != ENGRAM_ROW_DEAD;
  return (uint32_t)p.rows;
}

// Stable ranks of a tile's pairs by one digit.  Warp w holds pairs w*32*PER .. in order,
// pair (round r, lane l) at w*32*PER + 32 r + l; slots at or past n are left out.  On
// return place[r] is the pair's position among the tile's pairs sorted by digit, and
// s_start[d] the first position of digit d.
template <int PER>
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[PER], int n, int shift, int bits,
                                          uint16_t (*s_cnt)[kDigits], uint32_t *s_start, uint32_t *s_sum,
                                          uint32_t (&place)[PER]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mask = (1u << bits) - 1;
  uint4 *zero = reinterpret_cast<uint4 *>(s_cnt[warp]);
  for (int i = lane; i <= (int)mask / 8; i += 32) zero[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const bool have = warp * 32 * PER + 32 * r + lane < n;
    const uint32_t d = (key[r] >> shift) & mask;
    uint32_t same = __ballot_sync(0xffffffffu, have);  // the lanes with this digit, bit by bit
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      if (b == bits) break;
      const uint32_t set = __ballot_sync(0xffffffffu, d >> b & 1);
      same &= d >> b & 1 ? set : ~set;
    }
    const uint32_t before = __popc(same & ((1u << lane) - 1));
    if (have) {
      place[r] = s_cnt[warp][d] + before;
      __syncwarp(same);
      if (before == 0) s_cnt[warp][d] += (uint16_t)__popc(same);
    }
    __syncwarp();
  }
  __syncthreads();
  // Exclusive prefix over the warps of each digit (two a thread, added side by side: a
  // tile's counts fit 16 bits), then over the digits.
  uint32_t total = 0;
  if (2 * tid <= (int)mask) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      uint32_t *both = reinterpret_cast<uint32_t *>(s_cnt[w]) + tid;
      const uint32_t c = *both;
      *both = total;
      total += c;
    }
  }
  const uint32_t base = block_exclusive((total & 0xFFFF) + (total >> 16), s_sum);
  s_start[2 * tid] = base;
  s_start[2 * tid + 1] = base + (total & 0xFFFF);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < PER; ++r)
    if (warp * 32 * PER + 32 * r + lane < n) {
      const uint32_t d = (key[r] >> shift) & mask;
      place[r] += s_cnt[warp][d] + s_start[d];
    }
}

// The sort of up to kCountSort pairs: a pair's place is the number of pairs with a smaller
// key, or an equal one and an earlier position.  Each warp places 4 pairs, its lanes
// comparing them with 4 keys a load; positions are compared only inside the block's own 32
// pairs (before them equal keys count, behind them they do not).
constexpr int kCountThreads = 256, kCountOwn = 4, kCountPairs = kCountThreads / 32 * kCountOwn;

__global__ void __launch_bounds__(kCountThreads)
    count_sort_kernel(const __grid_constant__ EmbedGradParams p) {
  extern __shared__ uint4 s_key4[];
  uint32_t *s_key = reinterpret_cast<uint32_t *>(s_key4);
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)p.n;
  bool bad = false;
#pragma unroll 8
  for (int i = tid; i < (n + 3) / 4 * 4; i += kCountThreads)
    s_key[i] = i < n ? key_of(p, i, bad) : 0xFFFFFFFFu;  // the padding sorts behind everything
  if (bad && p.status && blockIdx.x == 0) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
  if (blockIdx.x == 0 && tid == 0) *p.long_count = 0;
  __syncthreads();
  const int first = blockIdx.x * kCountPairs;  // a multiple of 4, as are all the bounds below
  const int mine = first + warp * kCountOwn;
  uint32_t key[kCountOwn];
  int count[kCountOwn];
#pragma unroll
  for (int i = 0; i < kCountOwn; ++i) {
    key[i] = mine + i < n ? s_key[mine + i] : 0;
    count[i] = 0;
  }
  const int end = (n + 3) / 4, own = first / 4, after = min(end, own + kCountPairs / 4);
#pragma unroll 4
  for (int j = lane; j < own; j += 32) {
    const uint4 k = s_key4[j];
#pragma unroll
    for (int i = 0; i < kCountOwn; ++i)
      count[i] += (k.x <= key[i]) + (k.y <= key[i]) + (k.z <= key[i]) + (k.w <= key[i]);
  }
  for (int j = own + lane; j < after; j += 32) {
    const uint4 k = s_key4[j];
#pragma unroll
    for (int i = 0; i < kCountOwn; ++i) {
      const int at = mine + i - 4 * j;  // positions 4j .. 4j+3 against this pair's
      count[i] += (k.x < key[i] || (k.x == key[i] && at > 0)) + (k.y < key[i] || (k.y == key[i] && at > 1)) +
                  (k.z < key[i] || (k.z == key[i] && at > 2)) + (k.w < key[i] || (k.w == key[i] && at > 3));
    }
  }
#pragma unroll 4
  for (int j = after + lane; j < end; j += 32) {
    const uint4 k = s_key4[j];
#pragma unroll
    for (int i = 0; i < kCountOwn; ++i)
      count[i] += (k.x < key[i]) + (k.y < key[i]) + (k.z < key[i]) + (k.w < key[i]);
  }
#pragma unroll
  for (int i = 0; i < kCountOwn; ++i) {
    const int place = __reduce_add_sync(0xffffffffu, count[i]);
    if (lane == i && mine + i < n) {
      p.keys[place] = key[i];
      p.pos[place] = mine + i;
    }
  }
}

// ---- one pass of the sort of many pairs -----------------------------------------------

template <bool FIRST, int PER>
__global__ void __launch_bounds__(kSortThreads)
    count_digits_kernel(const __grid_constant__ EmbedGradParams p, const uint32_t *__restrict__ keys,
                        int shift) {
  __shared__ uint32_t s_cnt[kDigits];
  dependency_wait();
  const int tid = threadIdx.x;
  const uint32_t mask = (1u << p.digit_bits) - 1;
  for (int d = tid; d < kDigits; d += kSortThreads) s_cnt[d] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * (kSortThreads * PER);
  bool bad = false;
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int64_t i = base + r * kSortThreads + tid;
    if (i < p.n) {
      const uint32_t k = FIRST ? key_of(p, (uint32_t)i, bad) : __ldg(keys + i);
      atomicAdd(&s_cnt[(k >> shift) & mask], 1u);
    }
  }
  if (FIRST && bad && p.status) atomicOr(p.status, ENGRAM_FLAG_BAD_ROW);
  __syncthreads();
  for (int d = tid; d <= (int)mask; d += kSortThreads)
    p.counts[(int64_t)blockIdx.x << p.digit_bits | d] = s_cnt[d];
}

// counts[tile][digit] becomes its exclusive prefix sums over the tiles; the digits' totals go
// to `totals`.  A block takes 32 digits, a lane each; its warps take the tiles in as many
// contiguous parts: their sums first, then, from what comes before a part, its prefix.
constexpr int kScanThreads = 1024, kScanAhead = 8;
__global__ void __launch_bounds__(kScanThreads) scan_digits_kernel(uint32_t *counts, int64_t tiles, int32_t bits,
                                                                   uint32_t *totals, uint32_t *long_count) {
  __shared__ uint32_t s_sum[kScanThreads / 32][32];
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  const bool mine = d < 1 << bits;
  const int64_t per = (tiles + kScanThreads / 32 - 1) / (kScanThreads / 32);
  const int64_t first = warp * per, last = min(first + per, tiles);
  uint32_t *c = counts + d;
  uint32_t sum = 0;
  for (int64_t t = first; mine && t < last; t += kScanAhead) {
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (t + i < last) sum += c[(t + i) << bits];
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kScanThreads / 32; ++w) {
    const uint32_t v = s_sum[w][lane];
    before += w < warp ? v : 0;
    all += v;
  }
  for (int64_t t = first; mine && t < last; t += kScanAhead) {
    uint32_t v[kScanAhead];
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) v[i] = t + i < last ? c[(t + i) << bits] : 0;
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i)
      if (t + i < last) {
        c[(t + i) << bits] = before;
        before += v[i];
      }
  }
  if (mine && warp == 0) totals[d] = all;
  if (threadIdx.x == 0 && blockIdx.x == 0) *long_count = 0;
}

template <bool FIRST, int PER>
__global__ void __launch_bounds__(kSortThreads, 3)
    scatter_kernel(const __grid_constant__ EmbedGradParams p, const uint32_t *__restrict__ keys,
                   const uint32_t *__restrict__ poss, uint32_t *__restrict__ keys_out,
                   uint32_t *__restrict__ pos_out, int shift) {
  constexpr int kTile = kSortThreads * PER;
  extern __shared__ __align__(16) uint8_t s_all[];  // scatter_smem(PER)
  auto s_cnt = reinterpret_cast<uint16_t (*)[kDigits]>(s_all);
  uint32_t *s_start = reinterpret_cast<uint32_t *>(s_cnt + kSortWarps);
  uint32_t *s_key = s_start + kDigits;
  uint16_t *s_from = reinterpret_cast<uint16_t *>(s_key + kTile);
  __shared__ uint32_t s_sum[2][32];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mask = (1u << p.digit_bits) - 1;
  const int64_t base = (int64_t)blockIdx.x * kTile;
  const int n = (int)(p.n - base < kTile ? p.n - base : kTile);
  // What every digit has before it over all tiles, and this digit in the tiles before this one.
  uint32_t total[2], ahead[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 2 * tid + h;
    total[h] = d <= (int)mask ? __ldg(p.totals + d) : 0;
    ahead[h] = d <= (int)mask ? __ldg(p.counts + ((int64_t)blockIdx.x << p.digit_bits | d)) : 0;
  }
  uint32_t key[PER], place[PER];
  bool bad = false;
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = warp * 32 * PER + 32 * r + lane;
    key[r] = 0;
    if (i < n) key[r] = FIRST ? key_of(p, (uint32_t)(base + i), bad) : __ldg(keys + base + i);
  }
  rank_tile<PER>(key, n, shift, p.digit_bits, s_cnt, s_start, s_sum[0], place);
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = warp * 32 * PER + 32 * r + lane;
    if (i < n) {
      s_key[place[r]] = key[r];
      s_from[place[r]] = (uint16_t)i;
    }
  }
  // Where a digit of this tile goes, less its first position in the tile.
  const uint32_t to = block_exclusive(total[0] + total[1], s_sum[1]);
  s_start[2 * tid] = to + ahead[0] - s_start[2 * tid];
  s_start[2 * tid + 1] = to + total[0] + ahead[1] - s_start[2 * tid + 1];
  __syncthreads();
  uint32_t pos[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = r * kSortThreads + tid;
    if (i < n) {
      const uint32_t from = (uint32_t)base + s_from[i];
      pos[r] = FIRST ? from : __ldg(poss + from);
    }
  }
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = r * kSortThreads + tid;
    if (i < n) {
      const uint32_t k = s_key[i];
      const uint32_t at = s_start[(k >> shift) & mask] + i;
      keys_out[at] = k;
      pos_out[at] = pos[r];
    }
  }
}

constexpr size_t scatter_smem(int per) {
  return kSortWarps * kDigits * 2 + kDigits * 4 + (size_t)kSortThreads * per * 6;
}

// Both of the next two kernels' work for lists that one block reads quickly (1024 pairs: 9.2 us
// in all, by the two kernels 10.6).
constexpr int kRunsSmall = kCountSort;
__global__ void __launch_bounds__(kSortThreads) runs_small_kernel(const __grid_constant__ EmbedGradParams p) {
  __shared__ uint32_t s_sum[32];
  dependency_wait();
  constexpr int kEach = kRunsSmall / kSortThreads;  // at most, a multiple of 4
  const int n = (int)p.n, per = ((n + kSortThreads - 1) / kSortThreads + 3) / 4 * 4;
  const int e0 = threadIdx.x * per;
  uint32_t starts = 0;  // a bit an entry
  uint32_t before = e0 > 0 && e0 < n ? __ldg(p.keys + e0 - 1) : kNoKey;
#pragma unroll
  for (int i = 0; i < kEach; i += 4) {
    if (i < per && e0 + i < n) {
      const uint4 k4 = __ldg(reinterpret_cast<const uint4 *>(p.keys + e0 + i));
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (e0 + i + q < n && k[q] < (uint32_t)p.rows && k[q] != before) starts |= 1u << (i + q);
        before = k[q];
      }
    }
  }
  const uint32_t base = block_exclusive(__popc(starts), s_sum);
  for (int i = 0; i < per && e0 + i < n; ++i)  // chunks that start here (their length is 4 at least)
    if ((e0 + i) % p.chunk == 0) {
      const int c = (e0 + i) / p.chunk;
      p.run_base[c] = base + __popc(starts & ((1u << i) - 1));
      if (c % kRunGroup == 0) p.run_group[c / kRunGroup] = 0;
    }
  if (threadIdx.x == kSortThreads - 1) {
    *p.run_total = base + __popc(starts);
    *p.count_out = (int32_t)(base + __popc(starts));
  }
}

// Runs that start in a group of kRunGroup chunks, and before each of them in the group: a block
// a group, a warp a chunk.
__global__ void __launch_bounds__(kRunGroup * 32) count_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  __shared__ uint32_t s_count[kRunGroup];
  dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * kRunGroup + warp;
  const int64_t e0 = c * p.chunk, e1 = min(e0 + p.chunk, p.n);
  uint32_t mine = 0;
#pragma unroll 4
  for (int64_t e = e0 + lane; e < e1; e += 32) {
    const uint32_t k = __ldg(p.keys + e);
    mine += k < (uint32_t)p.rows && (e == 0 || __ldg(p.keys + e - 1) != k);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) s_count[warp] = mine;
  __syncthreads();
  if (warp != 0) return;
  const uint32_t v = lane < kRunGroup ? s_count[lane] : 0;
  uint32_t sum = v;
#pragma unroll
  for (int o = 1; o < kRunGroup; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane < kRunGroup && c + lane < p.chunks) p.run_base[c + lane] = sum - v;
  if (lane == kRunGroup - 1) p.run_group[blockIdx.x] = sum;
}

// run_group becomes its exclusive prefix sums; the number of runs goes to run_total.
__global__ void __launch_bounds__(1024) scan_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  __shared__ uint32_t s_sum[2][32];
  dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t groups = (p.chunks + kRunGroup - 1) / kRunGroup;
  uint32_t carry = 0;
  int buf = 0;
  for (int64_t i0 = 0; i0 < groups; i0 += 1024, buf ^= 1) {
    const uint32_t v = i0 + tid < groups ? p.run_group[i0 + tid] : 0;
    uint32_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) s_sum[buf][warp] = sum;
    __syncthreads();
    const uint32_t w = s_sum[buf][lane];  // every warp adds up the warps before it
    const uint32_t at = carry + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + sum - v;
    carry += __reduce_add_sync(0xffffffffu, w);
    if (i0 + tid < groups) p.run_group[i0 + tid] = at;
  }
  if (tid == 0) {
    *p.run_total = carry;
    *p.count_out = (int32_t)carry;
  }
}

// Runs that start before chunk c.
__device__ __forceinline__ int64_t runs_before(const EmbedGradParams &p, int64_t c) {
  return (int64_t)__ldg(p.run_base + c) + __ldg(p.run_group + c / kRunGroup);
}

// ---- sums of runs ------------------------------------------------------------------------

// A lane's columns: VEC: 8 neighbouring ones (16-byte accesses); else kLoose of them, a group's
// lanes apart, of which n lie in the row.  Three: one takes a third longer (40,674 pairs x 1278
// fp32 189 us, 152 with three), four leaves short lists with fewer lanes (3000 x 250: 31 us, 29).
constexpr int kLoose = 3;
template <bool VEC>
constexpr int kCols = VEC ? 8 : kLoose;

template <typename T, bool VEC>
struct Slice {  // as loaded
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *src, int, int) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
  }
  __device__ __forceinline__ void add_to(float (&acc)[8]) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
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
struct Slice<T, false> {
  T w[kLoose];
  __device__ __forceinline__ void load(const T *src, int apart, int n) {
#pragma unroll
    for (int i = 0; i < kLoose; ++i) w[i] = i < n ? __ldg(src + i * apart) : T(0);
  }
  __device__ __forceinline__ void add_to(float (&acc)[kLoose]) const {
#pragma unroll
    for (int i = 0; i < kLoose; ++i) {
      if constexpr (sizeof(T) == 4)
        acc[i] += w[i];
      else
        acc[i] += bf16_lo(w[i]);
    }
  }
};

// dst = scale * acc, or dst += scale * acc.
template <typename T, bool VEC>
__device__ __forceinline__ void write_row(T *dst, const float (&acc)[kCols<VEC>], int apart, int n, float scale,
                                          bool accumulate) {
  constexpr int V = kCols<VEC>;
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i >= n) continue;
      float f = acc[i] * scale;
      if constexpr (sizeof(T) == 4)
        dst[i * apart] = accumulate ? f + dst[i * apart] : f;
      else
        dst[i * apart] =
            __bfloat16_as_ushort(__float2bfloat16_rn(accumulate ? f + bf16_lo(dst[i * apart]) : f));
    }
  } else {
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
    if constexpr (sizeof(T) == 4) {
      __stcs(reinterpret_cast<float4 *>(dst), make_float4(f[0], f[1], f[2], f[3]));
      __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(f[4], f[5], f[6], f[7]));
    } else {
      __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                         pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void write_partial(float *dst, const float (&acc)[kCols<VEC>], int apart, int n) {
  if constexpr (VEC) {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kLoose; ++i)
      if (i < n) dst[i * apart] = acc[i];
  }
}

// The first of a lane's columns in a slab, and how many of them lie in the row.
template <bool VEC>
__device__ __forceinline__ int column_of(const EmbedGradParams &p, int slab, int in, int &n) {
  const int col = VEC ? (slab * p.group + in) * 8 : slab * p.group * kLoose + in;
  n = col >= p.D ? 0 : VEC ? 8 : (p.D - col + p.group - 1) / p.group;
  return col;
}

constexpr int kSumThreads = 128;

// A group's place: the chunk and the columns it works on.
struct Item {
  int64_t chunk;
  int slab, col, n, in;
};
template <bool VEC>
__device__ __forceinline__ Item item_of(const EmbedGradParams &p, int64_t group, int in) {
  Item it;
  it.chunk = group / p.slabs;
  it.slab = (int)(group - it.chunk * p.slabs);
  it.in = in;
  it.col = column_of<VEC>(p, it.slab, in, it.n);
  return it;
}

template <typename TY, typename TG, bool VEC, int U>
__device__ __forceinline__ void sum_chunk(const EmbedGradParams &p, const Item &it) {
  constexpr int V = kCols<VEC>;
  const int64_t C = p.chunk, e0 = it.chunk * C, e1 = min(e0 + C, p.n);
  const uint32_t rows = (uint32_t)p.rows;
  const bool mine = it.n > 0;
  const bool lead = it.slab == 0 && it.in == 0;
  const uint32_t first = __ldg(p.keys + e0), last = __ldg(p.keys + e1 - 1);
  const bool comes = e0 > 0 && __ldg(p.keys + e0 - 1) == first;
  const bool leaves = e1 < p.n && __ldg(p.keys + e1) == last;
  const bool through = comes && leaves && first == last;
  // A run that touches three chunks or more is summed in parts, one that touches two by the
  // chunk that it starts in.
  const bool long_in = comes && (through || (e0 - C >= 1 && __ldg(p.keys + e0 - C - 1) == first));
  const bool long_out = leaves && (through || (e0 + 2 * C < p.n && __ldg(p.keys + e0 + 2 * C) == last));
  int64_t run = 0;
  if (p.run_base) {
    run = runs_before(p, it.chunk) - comes;
    if (it.slab == 0) {  // ids beyond the distinct ones
      const int64_t count = __ldg(p.run_total);
      for (int64_t e = e0 + it.in; e < e1; e += p.group)
        if (e >= count) p.row_ids_out[e] = ENGRAM_ROW_DEAD;
    }
  }
  if (first >= rows) return;
  if (long_out && !through && lead && last < rows) p.long_list[atomicAdd(p.long_count, 1u)] = (uint32_t)it.chunk;
  const int64_t end = leaves && !long_out ? min(e0 + 2 * C, p.n) : e1;
  const bool skip = comes && !long_in;  // the first run is the chunk before's
  uint32_t cur = first;
  bool open = comes;
  const TY *dy = static_cast<const TY *>(p.dy) + it.col;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const auto flush = [&](bool out_part) {
    if (open && skip) return;
    if (open || out_part) {
      if (mine)
        write_partial<VEC>(p.partial + (it.chunk * 2 + (open ? 0 : 1)) * p.partial_stride + it.col, acc, p.group,
                           it.n);
    } else {
      const int64_t row = p.run_base ? run : cur;
      if (mine)
        write_row<TG, VEC>(static_cast<TG *>(p.grad) + row * p.grad_stride + it.col, acc, p.group, it.n, p.scale,
                           p.accumulate);
      if (p.run_base && lead) p.row_ids_out[run] = (int32_t)cur;
    }
  };
  // U entries at a time, the next ones' keys and positions on their way meanwhile.
  uint4 next_key[U / 4], next_pos[U / 4];
  const auto fetch = [&](int64_t e) {
#pragma unroll
    for (int i = 0; i < U / 4; ++i) {
      next_key[i] = __ldg(reinterpret_cast<const uint4 *>(p.keys + e) + i);
      next_pos[i] = __ldg(reinterpret_cast<const uint4 *>(p.pos + e) + i);
    }
  };
  fetch(e0);
  for (int64_t e = e0; e < end; e += U) {
    uint32_t key[U];
    Slice<TY, VEC> s[U];
    // past the chunk only its last run counts; kNoKey ends the walk
    const int in_chunk = (int)min(e1 - e, (int64_t)U), in_walk = (int)min(end - e, (int64_t)U);
#pragma unroll
    for (int i = 0; i < U / 4; ++i) {
      const uint32_t kk[4] = {next_key[i].x, next_key[i].y, next_key[i].z, next_key[i].w};
      const uint32_t pp[4] = {next_pos[i].x, next_pos[i].y, next_pos[i].z, next_pos[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = 4 * i + q;
        key[u] = u < in_chunk || (u < in_walk && kk[q] == last) ? kk[q] : kNoKey;
        if (mine && key[u] < rows && !(skip && key[u] == first)) {
          int64_t at = (int64_t)pp[q] * p.dy_id_stride;
          if (!p.dy_linear) {
            const uint32_t t = fast_div(pp[q], p.by_ids);
            at = t * p.dy_token_stride + (int64_t)(pp[q] - t * (uint32_t)p.n_ids) * p.dy_id_stride;
          }
          s[u].load(dy + at, p.group, it.n);
        }
      }
    }
    if (e + U < end) fetch(e + U);
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
      if (mine && !(open && skip)) s[u].add_to(acc);
    }
  }
  flush(long_out);
}

// p.zero_rows rows of a dense gradient (32 at most): those that no id names are zeroed.
template <typename TG, bool VEC>
__device__ __forceinline__ void zero_rows(const EmbedGradParams &p, int64_t r0) {
  const int lane = threadIdx.x & 31;
  // The first key >= r0: 32 probes at a time.
  int64_t lo = 0, hi = p.n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int less = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(p.keys + at) < (uint32_t)r0));
    if (less == 0) break;
    hi = min(lo + less * step, hi);
    lo += (less - 1) * step + 1;
  }
  // Which of the rows the keys from there on name, 32 keys at a time; behind a long run of
  // one row, a search of its own per row.
  const int64_t end = min(r0 + p.zero_rows, p.rows);
  uint32_t named = 0;
  bool done = false;
  for (int i = 0; i < 4 && !done; ++i, lo += 32) {
    const uint32_t k = lo + lane < p.n ? __ldg(p.keys + lo + lane) : kNoKey;
    named |= __reduce_or_sync(0xffffffffu, k < (uint32_t)end ? 1u << (k - (uint32_t)r0) : 0);
    done = __any_sync(0xffffffffu, k >= (uint32_t)end);
  }
  const int64_t row = r0 + lane;
  if (!done && row < end && !(named >> lane & 1)) {
    int64_t a = lo, b = p.n;  // the first key >= row
    while (a < b) {
      const int64_t mid = (a + b) >> 1;
      if (__ldg(p.keys + mid) < (uint32_t)row)
        a = mid + 1;
      else
        b = mid;
    }
    if (a < p.n && __ldg(p.keys + a) == (uint32_t)row) named |= 1u << lane;
  }
  const bool zero = row < end && !(named >> lane & 1);
  const uint32_t todo = __ballot_sync(0xffffffffu, zero);
  constexpr int kWord = VEC ? 16 / (int)sizeof(TG) : 1;  // values stored at once
  const uint32_t words = (uint32_t)p.D / kWord;
  TG *base = static_cast<TG *>(p.grad) + r0 * p.grad_stride;
  const auto clear = [](TG *dst) {
    if constexpr (VEC)
      __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(0, 0, 0, 0));
    else
      *dst = TG(0);
  };
  if (words >= 64) {  // wide rows: one after the other
    for (uint32_t left = todo; left; left &= left - 1) {
      TG *dst = base + (__ffs(left) - 1) * p.grad_stride;
      for (uint32_t c = lane; c < words; c += 32) clear(dst + c * kWord);
    }
  } else {  // narrow ones: their words through the lanes, whichever row they are in
#pragma unroll 4
    for (uint32_t i = lane; i < words * (uint32_t)p.zero_rows; i += 32) {
      const uint32_t r = words == 1 ? i : __umulhi(i, p.zero_magic);
      if (todo >> r & 1) clear(base + r * p.grad_stride + (i - r * words) * kWord);
    }
  }
}

template <typename TY, typename TG, bool VEC, int U>
__global__ void __launch_bounds__(kSumThreads) sum_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  dependency_wait();
  // Block b is zeroing block z if it is the z-th of them, spread evenly over the grid.
  const uint64_t b = blockIdx.x, all = p.sum_blocks + p.zero_blocks;
  const uint64_t z = b * p.zero_blocks / all;
  if ((b + 1) * p.zero_blocks / all > z) {
    const int64_t r0 = (z * (kSumThreads / 32) + (threadIdx.x >> 5)) * (int64_t)p.zero_rows;
    if (r0 < p.rows) zero_rows<TG, VEC>(p, r0);
    return;
  }
  const int64_t group = ((int64_t)(b - z) * kSumThreads + threadIdx.x) / p.group;
  const Item it = item_of<VEC>(p, group, threadIdx.x & (p.group - 1));
  if (it.chunk < p.chunks) sum_chunk<TY, TG, VEC, U>(p, it);
}

// ---- runs in parts ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;

// A block at a time takes a listed run and a slab of columns: each of its groups adds every
// groups-th part (the keys that end the run are loaded along with the parts), then the groups'
// sums are added up.
template <typename TG, bool VEC>
__global__ void __launch_bounds__(kJoinThreads) join_runs_kernel(const __grid_constant__ EmbedGradParams p) {
  constexpr int V = kCols<VEC>;
  extern __shared__ float s_part[];  // [groups][lanes a group * V]
  dependency_wait();
  const int G = p.group, groups = kJoinThreads / G;
  const int slot = threadIdx.x / G, in = threadIdx.x & (G - 1);
  const int64_t C = p.chunk, items = (int64_t)*p.long_count * p.slabs;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t listed = item / p.slabs;
    const int slab = (int)(item - listed * p.slabs);
    int n;
    const int col = column_of<VEC>(p, slab, in, n);
    const bool mine = n > 0;
    const int64_t chunk = __ldg(p.long_list + listed);
    const uint32_t key = __ldg(p.keys + (chunk + 2) * C);
    float acc[V] = {};
    bool more = true, any = false;
    for (int64_t i0 = slot; more; i0 += 4 * groups) {
      uint32_t k[4];
      Slice<float, VEC> s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * groups, c = chunk + i;
        k[u] = i == 0 ? key : (c < p.chunks ? __ldg(p.keys + c * C) : kNoKey);
        if (mine && c < p.chunks)
          s[u].load(p.partial + (c * 2 + (i == 0 ? 1 : 0)) * p.partial_stride + col, G, n);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        more = more && k[u] == key;
        any |= more;
        if (more && mine) s[u].add_to(acc);
      }
    }
    // The groups that had a part are the first ones; their sums meet as a tree.
    int active = __syncthreads_count(in == 0 && any);
    int half = 1;
    while (2 * half < active) half *= 2;
    for (; active > 1; active = half, half /= 2) {
      if (slot >= half && slot < active) {
#pragma unroll
        for (int i = 0; i < V; ++i) s_part[(slot * G + in) * V + i] = acc[i];
      }
      __syncthreads();
      if (slot + half < active) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += s_part[((slot + half) * G + in) * V + i];
      }
    }
    if (slot == 0) {
      const int64_t row = p.run_base ? runs_before(p, chunk + 1) - 1 : key;
      if (mine)
        write_row<TG, VEC>(static_cast<TG *>(p.grad) + row * p.grad_stride + col, acc, G, n, p.scale, p.accumulate);
      if (p.run_base && slab == 0 && in == 0) p.row_ids_out[row] = (int32_t)key;
    }
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------------------

int64_t sort_tiles(int64_t n) {
  const int64_t tile = kSortThreads * (n >= kLargeTiles ? kPerLarge : kPerSmall);
  return (n + tile - 1) / tile;
}

size_t round16(size_t x) { return (x + 15) / 16 * 16; }

// How the sums are cut: lanes a group, column slabs, chunk length.
struct Cut {
  int vec, group, slabs, chunk;
  int64_t chunks, stride;  // stride: columns of a partial sum's row
};
Cut cut_of(int64_t n, int D, bool vec) {
  Cut c;
  c.vec = vec ? 8 : kLoose;
  const int cols = (D + c.vec - 1) / c.vec;
  c.group = 1;
  while (c.group < 32 && c.group < cols) c.group *= 2;
  c.slabs = (cols + c.group - 1) / c.group;
  // Chunks long enough that what starts one is a small part of it, short enough that there
  // are several warps for every SM's schedulers (4096 pairs of 256 columns: 15.9 us, with
  // chunks of 64 34.2).
  c.chunk = 64;
  const int64_t warps = kSms * 48;
  while (c.chunk > 16 && (n + c.chunk - 1) / c.chunk * c.slabs * c.group / 32 < warps) c.chunk /= 2;
  // Short lists: shorter chunks still, while their partial sums stay under 2 MB; narrow rows not
  // so short, as a warp has many of their chunks and the runs that need joining slow it down
  // (3861 pairs of 16 columns, 574 rows: 35 us with chunks of 4, 23 with 8; 1024 distinct ones of
  // 256: 9.1 and 10.4).
  const int least = c.group < 16 ? 8 : 4;
  while (c.chunk > least && (n + c.chunk - 1) / c.chunk * c.slabs * c.group / 32 < warps / 8 &&
         (n / (c.chunk / 2) + 1) * 2 * (D + 8) * 4 <= (2 << 20))
    c.chunk /= 2;
  c.chunks = (n + c.chunk - 1) / c.chunk;
  c.stride = (D + 7) / 8 * 8;
  return c;
}

struct Layout {
  size_t keys[2], pos[2], counts, totals, run_base, run_group, long_list, partial, total;
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
  l.counts = take((size_t)sort_tiles(n) * kDigits * 4);
  l.totals = take(kDigits * 4);
  l.run_base = take((size_t)c.chunks * 4);
  l.run_group = take((size_t)(c.chunks / kRunGroup + 2) * 4);  // their number in front
  l.long_list = take((size_t)(c.chunks + 1) * 4);
  l.partial = take((size_t)c.chunks * 2 * c.stride * 4);
  l.total = at;
  return l;
}

template <typename TY, typename TG, bool VEC>
cudaError_t launch_sums(EmbedGradParams p, cudaStream_t stream) {
  constexpr int U = 4;
  const int64_t groups = p.chunks * p.slabs;
  p.sum_blocks = (groups * p.group + kSumThreads - 1) / kSumThreads;
  // Rows a warp of the zeroing blocks looks up: 32, or fewer wide ones, about 64 KB.
  p.zero_rows = 32;
  while (p.zero_rows > 1 && (int64_t)p.zero_rows * p.D * (int)sizeof(TG) > 65536) p.zero_rows /= 2;
  const uint32_t words = p.D / (VEC ? 16 / (int)sizeof(TG) : 1);
  p.zero_magic = (uint32_t)(((1ull << 32) + words - 1) / words);  // exact below 2^32 / words words
  const int64_t per = kSumThreads / 32 * p.zero_rows;
  p.zero_blocks = p.run_base || p.accumulate ? 0 : (p.rows + per - 1) / per;
  const int64_t blocks = p.sum_blocks + p.zero_blocks;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (blocks > 0) e = launch(sum_runs_kernel<TY, TG, VEC, U>, blocks, kSumThreads, 0, stream, 1, p);
  if (e != cudaSuccess || p.chunks < 3) return e;  // no run touches three chunks
  const int64_t most = p.chunks / 2 * p.slabs;     // a listed run has two chunks' borders at least
  return launch(join_runs_kernel<TG, VEC>, most < kSms * 3 ? most : kSms * 3, kJoinThreads,
                kJoinThreads * kCols<VEC> * sizeof(float), stream, 1, p);
}

template <typename TY, typename TG>
cudaError_t launch_typed(const EmbedGradParams &p, bool vec, cudaStream_t stream) {
  return vec ? launch_sums<TY, TG, true>(p, stream) : launch_sums<TY, TG, false>(p, stream);
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
  p.tiles = sort_tiles(p.n);
  p.counts = reinterpret_cast<uint32_t *>(w + l.counts);
  p.totals = reinterpret_cast<uint32_t *>(w + l.totals);
  p.run_base = sparse ? reinterpret_cast<uint32_t *>(w + l.run_base) : nullptr;
  p.run_total = reinterpret_cast<uint32_t *>(w + l.run_group);
  p.run_group = p.run_total + 1;
  p.long_count = reinterpret_cast<uint32_t *>(w + l.long_list);
  p.long_list = p.long_count + 1;
  p.partial = reinterpret_cast<float *>(w + l.partial);
  p.partial_stride = c.stride;
  p.group = c.group;
  p.slabs = c.slabs;
  p.chunk = c.chunk;
  p.chunks = c.chunks;
  int bits = 1;
  while (bits < 32 && ((uint64_t)p.rows >> bits) != 0) ++bits;  // keys are 0 .. rows
  p.passes = (bits + 9) / 10;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(w + l.keys[0]), reinterpret_cast<uint32_t *>(w + l.keys[1])};
  uint32_t *pos[2] = {reinterpret_cast<uint32_t *>(w + l.pos[0]), reinterpret_cast<uint32_t *>(w + l.pos[1])};
  cudaError_t e = cudaSuccess;
  p.keys = keys[0];
  p.pos = pos[0];
  if (p.n == 0) {
    if (sparse) return cudaMemsetAsync(p.count_out, 0, 4, stream);
  } else if (p.n <= kCountSort) {
    e = launch(count_sort_kernel, (p.n + kCountPairs - 1) / kCountPairs, kCountThreads,
               (size_t)(p.n + 3) / 4 * 16, stream, 1, p);
    if (e != cudaSuccess) return e;
  } else {
    const bool large = p.n >= kLargeTiles;
    if (large) {  // the only kernels over 48 KB
      static std::atomic<uint64_t> configured{0};
      if ((e = raise_smem_ceiling(scatter_kernel<true, kPerLarge>, configured)) != cudaSuccess) return e;
      static std::atomic<uint64_t> configured_next{0};
      if ((e = raise_smem_ceiling(scatter_kernel<false, kPerLarge>, configured_next)) != cudaSuccess) return e;
    }
    for (int pass = 0; pass < p.passes && e == cudaSuccess; ++pass) {
      const int shift = pass * p.digit_bits, in = pass & 1 ^ 1, out = pass & 1;
      const bool first = pass == 0;
      e = launch(large ? (first ? count_digits_kernel<true, kPerLarge> : count_digits_kernel<false, kPerLarge>)
                       : (first ? count_digits_kernel<true, kPerSmall> : count_digits_kernel<false, kPerSmall>),
                 p.tiles, kSortThreads, 0, stream, 1, p, keys[in], shift);
      if (e == cudaSuccess)
        e = launch(scan_digits_kernel, ((1 << p.digit_bits) + 31) / 32, kScanThreads, 0, stream, 1, p.counts,
                   p.tiles, p.digit_bits, p.totals, p.long_count);
      if (e == cudaSuccess)
        e = launch(large ? (first ? scatter_kernel<true, kPerLarge> : scatter_kernel<false, kPerLarge>)
                         : (first ? scatter_kernel<true, kPerSmall> : scatter_kernel<false, kPerSmall>),
                   p.tiles, kSortThreads, scatter_smem(large ? kPerLarge : kPerSmall), stream, 1, p, keys[in],
                   pos[in], keys[out], pos[out], shift);
    }
    if (e != cudaSuccess) return e;
    p.keys = keys[(p.passes - 1) & 1];
    p.pos = pos[(p.passes - 1) & 1];
  }
  if (sparse && p.n > 0 && p.n <= kRunsSmall) {
    if ((e = launch(runs_small_kernel, 1, kSortThreads, 0, stream, 1, p)) != cudaSuccess) return e;
  } else if (sparse && p.n > 0) {
    e = launch(count_runs_kernel, (p.chunks + kRunGroup - 1) / kRunGroup, kRunGroup * 32, 0, stream, 1, p);
    if (e == cudaSuccess) e = launch(scan_runs_kernel, 1, 1024, 0, stream, 1, p);
    if (e != cudaSuccess) return e;
  }
  if (dy_dtype == ENGRAM_DTYPE_F32)
    return grad_dtype == ENGRAM_DTYPE_F32 ? launch_typed<float, float>(p, vec, stream)
                                          : launch_typed<float, uint16_t>(p, vec, stream);
  return grad_dtype == ENGRAM_DTYPE_F32 ? launch_typed<uint16_t, float>(p, vec, stream)
                                        : launch_typed<uint16_t, uint16_t>(p, vec, stream);
}

}  // namespace engram

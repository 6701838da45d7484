// train_internal.cuh -- launch parameters and launchers of the training kernels
// (embedding lookup and gradient, FP8 quantisation and product, the gate's
// backward pass), shared with their C ABI layer (train_api.cu).
#pragma once

#include "engram_internal.cuh"

namespace engram {

constexpr int kSms = 152;  // of a GB300; grids are sized by it

inline size_t dtype_bytes(int dtype) { return dtype == ENGRAM_DTYPE_F32 ? 4 : 2; }

struct FastDiv {  // x / d as x * mul >> shift, for x < 2^31
  uint32_t mul, shift;
};
// Exact with m = ceil(2^(31 + l) / d), l = ceil(log2 d) (m < 2^32).
inline FastDiv fast_div_of(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  FastDiv f;
  f.shift = 31 + l;
  f.mul = (uint32_t)(((1ull << f.shift) + d - 1) / d);
  return f;
}
__device__ __forceinline__ uint32_t fast_div(uint32_t x, const FastDiv &f) {
  return (uint32_t)(((uint64_t)x * f.mul) >> f.shift);
}

struct EmbedParams {
  const int32_t *ids;
  const void *table;
  void *out;
  int32_t *status;
  int64_t n_tokens, ids_stride, rows, table_stride, out_token_stride, out_id_stride;
  int32_t n_ids, D;
  float scale;
  FastDiv by_ids;  // set by the launcher
};
cudaError_t launch_embed(const EmbedParams &p, int table_dtype, int out_dtype, bool pooled,
                         cudaStream_t stream);

struct EmbedGradParams {
  const int32_t *ids;
  const void *dy;
  void *grad;            // dense: [rows, D]; sparse: a row per distinct id
  int32_t *row_ids_out;  // sparse: [n], the distinct ids, then ENGRAM_ROW_DEAD
  int32_t *count_out;    // sparse: how many
  int32_t *status;
  int64_t n, ids_stride, rows, dy_token_stride, dy_id_stride, grad_stride;
  int32_t n_ids, D;
  float scale;
  bool accumulate;
  // set by the launcher
  FastDiv by_ids;
  bool dy_linear;              // dy rows are dy_id_stride apart throughout
  int32_t passes, digit_bits;  // of the sort
  int64_t tiles;
  uint32_t *keys, *pos, *counts, *totals;
  uint32_t *run_base;   // sparse: runs before each chunk in its group of chunks; else NULL
  uint32_t *run_group;  // runs before each group
  uint32_t *run_total;
  float *partial;      // [chunks][2][partial_stride]: a run open at the start, at the end
  uint32_t *long_count, *long_list;  // chunks in which a run of more than two chunks starts
  int64_t partial_stride, chunks, sum_blocks, zero_blocks;
  int32_t zero_rows;    // rows a warp of the zeroing blocks looks at
  uint32_t zero_magic;  // ceil(2^32 / words a row)
  int32_t group, slabs, chunk;  // lanes a group, column slabs, sorted ids a chunk
};
size_t embed_grad_workspace_bytes(int64_t n, int32_t D);
cudaError_t launch_embed_grad(EmbedGradParams p, int dy_dtype, int grad_dtype, void *workspace,
                              bool sparse, cudaStream_t stream);

struct GateGradParams {
  const float *k;
  const uint8_t *state;  // NULL: every token live
  const uint16_t *x, *dy;
  uint16_t *dx;
  void *dk;
  const float *alpha;
  float4 *partial;  // [kGateGradMaxBlocks]: each block's sums of g <dy_s, k>
  float *dalpha;
  int64_t T;
  int32_t D;
  float eps;
  float inv_D, inv_sqrt_D;  // set by the launcher, as are the rest
  int32_t group;            // lanes per narrow token
};
constexpr int kGateGradMaxBlocks = 4096;
cudaError_t launch_gate_grad(const GateGradParams &p, int dk_dtype, cudaStream_t stream);

struct QuantiseParams {
  const void *x;
  uint8_t *q, *s;    // NULL q: no row copy
  uint8_t *qt, *st;  // NULL qt: no transposed copy
  int32_t *status;
  int64_t wait_limit_ns;
  int64_t M, K, x_stride, q_stride, qt_stride;
  int32_t block_rows;  // 1 or ENGRAM_FP8_BLOCK
  bool withhold;       // test hook, set by the launcher: a block's first copy is never issued
};
cudaError_t launch_quantise(const QuantiseParams &p, int dtype, cudaStream_t stream);

struct MatmulParams {
  const uint8_t *a, *a_scale, *b, *b_scale;
  void *out;
  int32_t *status;
  int64_t M, N, K, a_stride, b_stride, out_stride;
  int32_t a_block, b_block;  // rows sharing a scale: 1 or ENGRAM_FP8_BLOCK
};
cudaError_t launch_fp8_matmul(const MatmulParams &p, int out_dtype, cudaStream_t stream);

}  // namespace engram

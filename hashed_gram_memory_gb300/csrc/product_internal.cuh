// product_internal.cuh -- launch parameters and launchers of the 16-bit product and of what is
// built on it (its gradient, the orthogonalised update), shared with their C ABI layer
// (product_api.cu).
#pragma once

#include "train_internal.cuh"

namespace engram {

constexpr int kTypeF16 = 2;  // beside ENGRAM_DTYPE_*: values inside the library

// A 16-bit operand [rows, K]: element (r, k) at r * stride + k, or with `t` at k * stride + r.
// 16-byte aligned, stride and batch a multiple of 8 elements.
struct Operand {
  const void *p;
  int64_t stride, batch;  // batch: elements between matrices
  bool t;
};

// A value [M, N] per matrix, element (m, n) at m * stride + n; NULL: not there.
struct Plane {
  void *p;
  int64_t stride, batch;
  int32_t type;  // ENGRAM_DTYPE_* or kTypeF16
};

// out = act(scale * a b^T + bias) + residual_scale * residual, pre = what act is taken of; for
// `count` matrices.
struct ProductParams {
  Operand a, b;
  bool f16;  // operands: f16, else bf16
  bool a_two;  // a is the sum of two matrices, a.batch elements apart (count is 1)
  int64_t M, N, K, count;
  float scale, residual_scale;
  Plane out, residual, pre;
  const void *bias;
  int32_t bias_type, act;
  // a and b are one matrix and so out is symmetric (as must be residual): the products on one
  // side of the diagonal are computed, and written on both; out and residual are fp16, their
  // rows on 16-byte boundaries
  bool symmetric;
  // The iteration's products (fp16 operands and residual): the diagonals of the square matrices stay
  // fp32, [count][diag_batch] each, diag_batch a multiple of 64.  With D = diag_in residual (m, n) counts
  // residual_scale + diag_by (D[m] + D[n]) times, of which D has the rows' or the columns' or both;
  // diag_out (NULL: none) receives what out has at (m, m), times diag_scale, and (residual_scale + diag_by
  // D[m]) D[m], and there out becomes zero.
  bool newton, diag_rows, diag_columns;
  const float *diag_in;
  float *diag_out;
  int64_t diag_batch;
  float diag_by, diag_scale;
  int32_t *status;
};
cudaError_t launch_product(const ProductParams &p, cudaStream_t stream);
// Two products that do not depend on one another, in one launch where that is faster.
cudaError_t launch_products(const ProductParams &p0, const ProductParams &p1, cudaStream_t stream);

// The product for up to 16 rows of a (product_few.cu), which launch_product takes where it can.
bool few_rows_supported(const ProductParams &p);
cudaError_t launch_few_rows(const ProductParams &p, cudaStream_t stream);

// Copies of [rows, cols] 16-bit values from rows src_stride apart to rows dst_stride apart (a
// multiple of 8, dst 16-byte aligned).
struct Packed {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_stride, dst_stride, rows, cols;
};
struct PackParams {
  Packed part[2];
  int32_t count;
};
cudaError_t launch_pack(const PackParams &p, cudaStream_t stream);

// dz = dy * act'(pre), rounded to bf16, what that rounding left, rounded again, and dz's column sums
// before any rounding.
struct ActGradParams {
  const void *dy, *pre;  // pre NULL without an activation
  void *dz;              // bf16 [M, N], dz_stride a multiple of 8, or NULL
  void *dz_rest;         // the same, or NULL
  float *dbias;          // [N] or NULL
  float *partial;        // act_grad_partial_bytes()
  int64_t M, N, dy_stride, pre_stride, dz_stride;
  int32_t dy_type, pre_type, act;
  bool accumulate;  // dbias is added to
  // set by the launcher
  int32_t slabs, col_blocks, lanes, threads;
  int64_t slab_rows;
};
size_t act_grad_partial_bytes(int64_t M, int64_t N);
cudaError_t launch_act_grad(ActGradParams p, cudaStream_t stream);

// Newton-Schulz on `count` matrices [M, N].
struct OrthogonaliseParams {
  Plane g, momentum, out;  // momentum.p NULL: none
  int64_t M, N, count;
  float beta, eps, scale, a, b, c;
  int32_t steps;
  bool nesterov;
  int32_t *status;
};
size_t orthogonalise_workspace_bytes(int64_t M, int64_t N, int64_t count);
cudaError_t launch_orthogonalise(const OrthogonaliseParams &p, void *workspace, cudaStream_t stream);
// The same in one launch without a workspace (orthogonalise_small.cu), which launch_orthogonalise
// takes where it can.
bool orthogonalise_small_supported(const OrthogonaliseParams &p);
cudaError_t launch_orthogonalise_small(const OrthogonaliseParams &p, cudaStream_t stream);

}  // namespace engram

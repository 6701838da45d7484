// product_api.cu -- the extern "C" entry points of the 16-bit product, its gradient and the
// orthogonalised update: argument validation on the host, the device check and the launches.
#include <math.h>

#include "product_internal.cuh"

namespace {

using engram::dtype_bytes;
using engram::Operand;
using engram::Plane;
using engram::set_error;

constexpr int64_t kMost = INT32_MAX - 256;  // tile origins stay in 32 bits
constexpr int64_t kMostStride = (int64_t)1 << 38;  // of the copies' descriptors, in elements

engram_status ok() { return set_error(ENGRAM_OK, "%s", ""); }

engram_status launched(const char *what, cudaError_t e) {
  if (e != cudaSuccess)
    return set_error(ENGRAM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return ok();
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool dtype_ok(int32_t d) { return d == ENGRAM_DTYPE_BF16 || d == ENGRAM_DTYPE_F32; }

bool act_ok(int32_t a) { return a >= ENGRAM_ACT_NONE && a <= ENGRAM_ACT_GELU; }

// A buffer of a call: its bytes from the first to one past the last.
struct Span {
  const void *p;
  uint64_t n;
};
Span span_of(const void *p, int64_t rows, int64_t stride, int64_t cols, int64_t bytes) {
  return Span{p, p && rows > 0 ? (uint64_t)((rows - 1) * stride + cols) * bytes : 0};
}
bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

// A 16-bit operand [rows, K] as the caller has it.
struct Given {
  const uint16_t *p;
  int64_t stride;
  bool t;
  int64_t rows, K;
  int64_t outer() const { return t ? K : rows; }
  int64_t inner() const { return t ? rows : K; }
  Span span() const { return span_of(p, outer(), stride, inner(), 2); }
  bool valid() const {
    return p && aligned(p, 2) && (outer() == 1 || (stride >= inner() && stride <= kMostStride));
  }
  // The tensor copies read it where it is.
  bool direct() const { return aligned(p, 16) && (outer() == 1 || stride % 8 == 0); }
  int64_t packed_stride() const { return (inner() + 7) / 8 * 8; }
  size_t packed_bytes() const {
    return direct() ? 0 : (size_t)(outer() * packed_stride() * 2 + 255) / 256 * 256;
  }
};

// The operands for the products, as they are or their copies in the workspace (one launch for both).
cudaError_t operands_of(const Given *g[2], uint8_t *&scratch, Operand out[2], cudaStream_t stream) {
  engram::PackParams pack{};
  for (int i = 0; i < 2; ++i) {
    if (!g[i]) continue;
    out[i] = Operand{g[i]->p, g[i]->stride, 0, g[i]->t};
    if (g[i]->direct()) continue;
    engram::Packed &k = pack.part[pack.count++];
    k.src = g[i]->p;
    k.src_stride = g[i]->outer() > 1 ? g[i]->stride : 0;
    k.dst = reinterpret_cast<uint16_t *>(scratch);
    k.dst_stride = g[i]->packed_stride();
    k.rows = g[i]->outer();
    k.cols = g[i]->inner();
    out[i].p = scratch;
    out[i].stride = k.dst_stride;
    scratch += g[i]->packed_bytes();
  }
  return pack.count ? engram::launch_pack(pack, stream) : cudaSuccess;
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 1 && K >= 1 && M <= kMost && N <= kMost && K <= kMost;
}

// A plane [rows, cols] that a call writes (or reads, where rows may repeat: least stride 0).
bool plane_ok(const void *p, int32_t type, int64_t rows, int64_t stride, int64_t least) {
  return aligned(p, dtype_bytes(type)) && (rows <= 1 || (stride >= least && stride <= kMostStride));
}

// dz, the operand that the gradient's two products share, has to be made: it is not dy, or the
// tensor copies cannot read dy where it is (rows that repeat among them).
bool makes_dz(const Given &dy, int32_t dy_dtype, int32_t act) {
  return act != ENGRAM_ACT_NONE || dy_dtype != ENGRAM_DTYPE_BF16 || !dy.direct() ||
         (dy.rows > 1 && dy.stride < dy.K);
}
// dz has to be two matrices: of fp32 outputs, where it is not bf16 to begin with.
bool two_of_dz(const void *da, int32_t da_dtype, const void *db, int32_t db_dtype, int32_t dy_dtype, int32_t act) {
  return ((da && da_dtype == ENGRAM_DTYPE_F32) || (db && db_dtype == ENGRAM_DTYPE_F32)) &&
         (act != ENGRAM_ACT_NONE || dy_dtype != ENGRAM_DTYPE_BF16);
}
int64_t dz_stride_of(int64_t N) { return N > 512 ? (N + 63) / 64 * 64 : (N + 7) / 8 * 8; }
size_t dz_bytes(int64_t M, int64_t N) { return (size_t)(M * dz_stride_of(N) * 2 + 255) / 256 * 256; }

}  // namespace

extern "C" {

ENGRAM_API size_t engram_matmul_workspace_bytes(const engram_matmul_args *args) {
  if (!args || !sizes_ok(args->M, args->N, args->K)) return 0;
  return Given{args->a, args->a_stride, args->a_trans != 0, args->M, args->K}.packed_bytes() +
         Given{args->b, args->b_stride, args->b_trans != 0, args->N, args->K}.packed_bytes();
}

ENGRAM_API engram_status engram_matmul(const engram_matmul_args *args, void *workspace, size_t workspace_bytes,
                                       int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_matmul");
  const char *fn = "engram_matmul";
  if (!args) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const auto [a, a_stride, b, b_stride, M, N, K, bias, residual, residual_stride, pre, pre_stride, out, out_stride,
              a_trans, b_trans, activation, bias_dtype, residual_dtype, pre_dtype, out_dtype, scale] = *args;
  if (!sizes_ok(M, N, K))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: M >= 0, N >= 1 and K >= 1, all under 2^31 - 256", fn);
  if (!act_ok(activation)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown activation", fn);
  if (!dtype_ok(out_dtype) || (bias && !dtype_ok(bias_dtype)) || (residual && !dtype_ok(residual_dtype)) ||
      (pre && !dtype_ok(pre_dtype)))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (M == 0) return ok();
  const Given ga{a, a_stride, a_trans != 0, M, K}, gb{b, b_stride, b_trans != 0, N, K};
  if (!ga.valid() || !gb.valid())
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: a or b NULL or misaligned, or its stride under a row's width or over 2^38", fn);
  if (!out || !plane_ok(out, out_dtype, M, out_stride, N))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out NULL or misaligned, or its stride under N", fn);
  if (pre && !plane_ok(pre, pre_dtype, M, pre_stride, N))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: pre misaligned, or its stride under N", fn);
  if (residual && !plane_ok(residual, residual_dtype, M, residual_stride, 0))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: residual misaligned, or its stride negative", fn);
  if ((bias && !aligned(bias, dtype_bytes(bias_dtype))) || !aligned(status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: bias or status misaligned", fn);
  const size_t need = ga.packed_bytes() + gb.packed_bytes();
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: rows off 16-byte boundaries are copied: workspace NULL, not 16-byte aligned or under "
                     "%zu bytes",
                     fn, need);
  // The residual may be out itself: each value is read before it is written.
  const bool in_place =
      residual == out && residual_dtype == out_dtype && (M == 1 || residual_stride == out_stride);
  const Span outs[3] = {span_of(out, M, out_stride, N, dtype_bytes(out_dtype)),
                        span_of(pre, M, pre_stride, N, pre ? dtype_bytes(pre_dtype) : 0),
                        {need ? workspace : nullptr, need}};
  const Span res = span_of(residual, M, residual_stride, N, residual ? dtype_bytes(residual_dtype) : 0);
  const Span ins[5] = {ga.span(), gb.span(), {bias, bias ? (uint64_t)N * dtype_bytes(bias_dtype) : 0}, {status, 4},
                       res};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i)
      if (!(o == 0 && i == 4 && in_place) && overlap(outs[o], ins[i]))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  engram_status st = engram::check_sm103();
  if (st != ENGRAM_OK) return st;
  engram::ProductParams p{};
  uint8_t *scratch = static_cast<uint8_t *>(workspace);
  const Given *given[2] = {&ga, &gb};
  Operand operands[2];
  const cudaError_t e = operands_of(given, scratch, operands, (cudaStream_t)stream);
  if (e != cudaSuccess) return launched("engram_matmul launch", e);
  p.a = operands[0];
  p.b = operands[1];
  p.M = M;
  p.N = N;
  p.K = K;
  p.count = 1;
  p.scale = scale;
  p.residual_scale = 1.f;
  p.out = Plane{out, out_stride, 0, out_dtype};
  p.residual = Plane{const_cast<void *>(residual), residual_stride, 0, residual_dtype};
  p.pre = Plane{pre, pre_stride, 0, pre_dtype};
  p.bias = bias;
  p.bias_type = bias_dtype;
  p.act = activation;
  p.status = status;
  return launched("engram_matmul launch", engram::launch_product(p, (cudaStream_t)stream));
}

ENGRAM_API size_t engram_matmul_grad_workspace_bytes(const engram_matmul_grad_args *args) {
  if (!args) return 0;
  const engram_matmul_grad_args &g = *args;
  if (!sizes_ok(g.M, g.N, g.K) || g.M == 0) return 0;
  size_t bytes = 0;
  const Given gy{static_cast<const uint16_t *>(g.dy), g.dy_stride, false, g.M, g.N};
  if ((g.da || g.db) && makes_dz(gy, g.dy_dtype, g.activation))
    bytes += dz_bytes(g.M, g.N) << two_of_dz(g.da, g.da_dtype, g.db, g.db_dtype, g.dy_dtype, g.activation);
  if (g.dbias) bytes += (engram::act_grad_partial_bytes(g.M, g.N) + 255) / 256 * 256;
  if (g.db) bytes += Given{g.a, g.a_stride, g.a_trans != 0, g.M, g.K}.packed_bytes();
  if (g.da) bytes += Given{g.b, g.b_stride, g.b_trans != 0, g.N, g.K}.packed_bytes();
  return bytes;
}

ENGRAM_API engram_status engram_matmul_grad(const engram_matmul_grad_args *args, void *workspace,
                                            size_t workspace_bytes, int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_matmul_grad");
  const char *fn = "engram_matmul_grad";
  const cudaStream_t s = (cudaStream_t)stream;
  if (!args) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const auto [dy, dy_stride, a, a_stride, b, b_stride, M, N, K, given_pre, pre_stride, da, da_stride, db, db_stride,
              dbias, a_trans, b_trans, activation, dy_dtype, pre_dtype, da_dtype, db_dtype, accumulate, scale] = *args;
  if (!sizes_ok(M, N, K))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: M >= 0, N >= 1 and K >= 1, all under 2^31 - 256", fn);
  if (!act_ok(activation)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown activation", fn);
  const void *pre = activation == ENGRAM_ACT_NONE ? nullptr : given_pre;
  if (!da && !db && !dbias && M > 0) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: no gradient is asked for", fn);
  if (!dtype_ok(dy_dtype) || (pre && !dtype_ok(pre_dtype)) || (da && !dtype_ok(da_dtype)) ||
      (db && !dtype_ok(db_dtype)))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (db && !plane_ok(db, db_dtype, N, db_stride, K))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: db misaligned, or its stride under K", fn);
  if (!aligned(dbias, 4) || !aligned(status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: dbias or status misaligned", fn);
  if (M > 0) {
    if (!dy || !plane_ok(dy, dy_dtype, M, dy_stride, 0))
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: dy NULL or misaligned, or its stride negative", fn);
    if (activation != ENGRAM_ACT_NONE && (!pre || !plane_ok(pre, pre_dtype, M, pre_stride, 0)))
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: pre NULL or misaligned, or its stride negative", fn);
    if (da && !plane_ok(da, da_dtype, M, da_stride, K))
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: da misaligned, or its stride under K", fn);
  }
  const Given ga{a, a_stride, a_trans != 0, M, K}, gb{b, b_stride, b_trans != 0, N, K};
  if (M > 0 && ((db && !ga.valid()) || (da && !gb.valid())))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: a or b NULL or misaligned, or its stride under a row's width or over 2^38", fn);
  Given gy{static_cast<const uint16_t *>(dy), dy_stride, false, M, N};
  const bool dz = (da || db) && M > 0 && makes_dz(gy, dy_dtype, activation);
  const bool two = dz && two_of_dz(da, da_dtype, db, db_dtype, dy_dtype, activation);
  const int64_t between = (int64_t)dz_bytes(M, N) / 2;  // elements from dz to what its rounding left
  const size_t need = engram_matmul_grad_workspace_bytes(args);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: workspace NULL, not 16-byte aligned or under %zu bytes", fn, need);
  const Span outs[4] = {span_of(da, M, da_stride, K, da ? dtype_bytes(da_dtype) : 0),
                        span_of(db, N, db_stride, K, db ? dtype_bytes(db_dtype) : 0),
                        {dbias, (uint64_t)N * 4},
                        {need ? workspace : nullptr, need}};
  const Span ins[5] = {span_of(dy, M, dy_stride, N, dtype_bytes(dy_dtype)),
                       span_of(pre, M, pre_stride, N, pre ? dtype_bytes(pre_dtype) : 0),
                       db ? ga.span() : Span{nullptr, 0}, da ? gb.span() : Span{nullptr, 0}, {status, 4}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(outs[o], ins[i])) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  engram_status st = engram::check_sm103();
  if (st != ENGRAM_OK) return st;
  cudaError_t e = cudaSuccess;
  if (M == 0) {
    if (db && !accumulate)
      e = cudaMemset2DAsync(db, db_stride * dtype_bytes(db_dtype), 0, K * dtype_bytes(db_dtype), N, s);
    if (e == cudaSuccess && dbias && !accumulate) e = cudaMemsetAsync(dbias, 0, (size_t)N * 4, s);
    return launched(fn, e);
  }
  uint8_t *scratch = static_cast<uint8_t *>(workspace);
  if (dz || dbias) {
    engram::ActGradParams g{};
    g.dy = dy;
    g.pre = pre;
    g.dbias = dbias;
    g.M = M;
    g.N = N;
    g.dy_stride = M > 1 ? dy_stride : 0;
    g.pre_stride = M > 1 ? pre_stride : 0;
    g.dy_type = dy_dtype;
    g.pre_type = pre ? pre_dtype : ENGRAM_DTYPE_BF16;
    g.act = activation;
    g.accumulate = accumulate != 0;
    if (dz) {
      g.dz = scratch;
      g.dz_stride = dz_stride_of(N);
      gy = Given{reinterpret_cast<uint16_t *>(scratch), g.dz_stride, false, M, N};
      scratch += dz_bytes(M, N);
      if (two) {
        g.dz_rest = scratch;
        scratch += dz_bytes(M, N);
      }
    }
    if (dbias) {
      g.partial = reinterpret_cast<float *>(scratch);
      scratch += (engram::act_grad_partial_bytes(M, N) + 255) / 256 * 256;
    }
    if ((e = engram::launch_act_grad(g, s)) != cudaSuccess) return launched(fn, e);
  }
  const Given *given[2] = {db ? &ga : nullptr, da ? &gb : nullptr};
  Operand operands[2] = {};
  if ((e = operands_of(given, scratch, operands, s)) != cudaSuccess) return launched(fn, e);
  const Operand &oa = operands[0], &ob = operands[1];
  engram::ProductParams pa{}, pb{};
  pa.count = 1;
  pa.scale = scale;
  pa.residual_scale = 1.f;
  pa.status = status;
  pb = pa;
  if (da) {  // rows of dz by the columns of b, over N
    pa.a = Operand{gy.p, gy.stride, between, false};
    pa.a_two = two && da_dtype == ENGRAM_DTYPE_F32;
    pa.b = Operand{ob.p, ob.stride, 0, !ob.t};
    pa.M = M;
    pa.N = K;
    pa.K = N;
    pa.out = Plane{da, da_stride, 0, da_dtype};
  }
  if (db) {  // columns of dz by the columns of a, over M
    pb.a = Operand{gy.p, gy.stride, between, true};
    pb.a_two = two && db_dtype == ENGRAM_DTYPE_F32;
    pb.b = Operand{oa.p, oa.stride, 0, !oa.t};
    pb.M = N;
    pb.N = K;
    pb.K = M;
    pb.out = Plane{db, db_stride, 0, db_dtype};
    if (accumulate) pb.residual = pb.out;
  }
  if (da && db)
    e = engram::launch_products(pa, pb, s);
  else if (da || db)
    e = engram::launch_product(da ? pa : pb, s);
  return launched(fn, e);
}

ENGRAM_API size_t engram_orthogonalise_workspace_bytes(int64_t count, int64_t M, int64_t N) {
  if (count < 0 || M < 1 || N < 1 || M > kMost || N > kMost) return 0;
  return engram::orthogonalise_workspace_bytes(M, N, count);
}

ENGRAM_API engram_status engram_orthogonalise(const void *g, int32_t g_dtype, int64_t count, int64_t M, int64_t N,
                                              int64_t g_batch, int64_t g_stride, float *momentum,
                                              int64_t momentum_batch, int64_t momentum_stride, float beta,
                                              int32_t nesterov, int32_t steps, float coeff_a, float coeff_b,
                                              float coeff_c, float scale, float eps, uint16_t *out,
                                              int64_t out_batch, int64_t out_stride, void *workspace,
                                              size_t workspace_bytes, int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_orthogonalise");
  const char *fn = "engram_orthogonalise";
  if (count < 0 || M < 1 || N < 1 || M > kMost || N > kMost || count > 65535)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: count in [0, 65535], M and N in [1, 2^31 - 256)", fn);
  if (!dtype_ok(g_dtype)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown g dtype", fn);
  if (steps < 1 || steps > 64) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: steps must be in [1, 64]", fn);
  if (!(fabsf(coeff_a) <= 16.f) || !(fabsf(coeff_b) <= 16.f) || !(fabsf(coeff_c) <= 16.f))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: coefficients must be in [-16, 16]", fn);
  if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(scale) || !isfinite(beta))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, scale and beta finite", fn);
  if (count == 0) return ok();
  const auto plane = [&](const void *p, int64_t type, int64_t batch, int64_t stride) {
    return p && aligned(p, dtype_bytes((int)type)) && (M == 1 || (stride >= N && stride <= kMostStride)) &&
           (count == 1 || (batch >= (M - 1) * (M == 1 ? 0 : stride) + N && batch <= kMostStride));
  };
  if (!plane(g, g_dtype, g_batch, g_stride))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: g NULL or misaligned, or its rows or matrices overlap", fn);
  if (momentum && !plane(momentum, ENGRAM_DTYPE_F32, momentum_batch, momentum_stride))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: momentum misaligned, or its rows or matrices overlap", fn);
  if (!plane(out, ENGRAM_DTYPE_BF16, out_batch, out_stride))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out NULL or misaligned, or its rows or matrices overlap", fn);
  if (!aligned(status, 4)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: status misaligned", fn);
  const size_t need = engram_orthogonalise_workspace_bytes(count, M, N);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: workspace NULL, not 16-byte aligned or under %zu bytes", fn, need);
  const auto whole = [&](const void *p, int64_t batch, int64_t stride, int64_t bytes) {
    const int64_t one = (M - 1) * stride + N;
    return span_of(p, count, batch, one, bytes);
  };
  const Span outs[3] = {whole(out, out_batch, out_stride, 2), whole(momentum, momentum_batch, momentum_stride, 4),
                        {workspace, need}};
  const Span ins[2] = {whole(g, g_batch, g_stride, dtype_bytes(g_dtype)), {status, 4}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 2; ++i)
      if (overlap(outs[o], ins[i])) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  engram_status st = engram::check_sm103();
  if (st != ENGRAM_OK) return st;
  engram::OrthogonaliseParams p{};
  p.g = Plane{const_cast<void *>(g), g_stride, g_batch, g_dtype};
  p.momentum = Plane{momentum, momentum_stride, momentum_batch, ENGRAM_DTYPE_F32};
  p.out = Plane{out, out_stride, out_batch, ENGRAM_DTYPE_BF16};
  p.M = M;
  p.N = N;
  p.count = count;
  p.beta = beta;
  p.eps = eps;
  p.scale = scale;
  p.a = coeff_a;
  p.b = coeff_b;
  p.c = coeff_c;
  p.steps = steps;
  p.nesterov = nesterov != 0;
  p.status = status;
  return launched("engram_orthogonalise launch",
                  engram::launch_orthogonalise(p, workspace, (cudaStream_t)stream));
}

}  // extern "C"

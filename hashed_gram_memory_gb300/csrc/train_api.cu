// train_api.cu -- the extern "C" entry points of the training calls: argument
// validation on the host, the device check and the launches.
#include <math.h>

#include "train_internal.cuh"

namespace {

using engram::dtype_bytes;
using engram::set_error;

engram_status ok() { return set_error(ENGRAM_OK, "%s", ""); }

engram_status launched(const char *what, cudaError_t e) {
  if (e != cudaSuccess)
    return set_error(ENGRAM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return ok();
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}

bool dtype_ok(int32_t d) { return d == ENGRAM_DTYPE_BF16 || d == ENGRAM_DTYPE_F32; }

// Elements from the first to one past the last of an [n, m, width] view.
int64_t extent(int64_t n, int64_t stride_n, int64_t m, int64_t stride_m, int64_t width) {
  return n > 0 && m > 0 ? (n - 1) * stride_n + (m - 1) * stride_m + width : 0;
}

// The checks of ids [n_tokens, n_ids] shared by the embedding calls.
engram_status check_ids(const char *fn, const int32_t *ids, int64_t n_tokens, int32_t n_ids,
                        int64_t ids_stride, int64_t rows, int32_t D, const int32_t *status) {
  if (n_tokens < 0 || n_ids < 1 || n_tokens > INT32_MAX / n_ids)
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: n_tokens >= 0, n_ids >= 1 and n_tokens * n_ids <= 2^31-1", fn);
  if (rows < 1 || rows > INT32_MAX)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: rows must be in [1, 2^31-1]", fn);
  if (D < 1 || D > ENGRAM_MAX_EMBED_D)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: D must be in [1, %d]", fn, ENGRAM_MAX_EMBED_D);
  if (n_tokens > 0 && !ids) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: ids is NULL", fn);
  if (!aligned(ids, 4) || !aligned(status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: int32 pointers must be 4-byte aligned", fn);
  if (n_tokens > 1 && ids_stride < n_ids)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: ids_stride is under n_ids", fn);
  return ENGRAM_OK;
}

}  // namespace

extern "C" {

ENGRAM_API engram_status engram_embed(const int32_t *ids, int64_t n_tokens, int32_t n_ids,
                                      int64_t ids_stride, const void *table, int32_t table_dtype,
                                      int64_t rows, int32_t D, int64_t table_stride, float scale,
                                      int32_t pooled, void *out, int32_t out_dtype,
                                      int64_t out_token_stride, int64_t out_id_stride,
                                      int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_embed");
  const char *fn = "engram_embed";
  engram_status st = check_ids(fn, ids, n_tokens, n_ids, ids_stride, rows, D, status);
  if (st != ENGRAM_OK) return st;
  if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (!table || !aligned(table, dtype_bytes(table_dtype)) || (rows > 1 && table_stride < D))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: table NULL or misaligned, or its stride under D", fn);
  const int64_t per = pooled ? 1 : n_ids;
  // The output rows must not share elements: either ids inside tokens or the other way round.
  const bool inner = out_id_stride >= D && out_token_stride >= (per - 1) * out_id_stride + D;
  const bool outer = out_token_stride >= D && out_id_stride >= (n_tokens - 1) * out_token_stride + D;
  if (per > 1 ? !(inner || (n_tokens <= 1 && out_id_stride >= D) || outer)
              : (n_tokens > 1 && out_token_stride < D))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output rows overlap (strides)", fn);
  if (n_tokens == 0) return ok();
  if (!out || !aligned(out, dtype_bytes(out_dtype)))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out NULL or misaligned", fn);
  const size_t ob = extent(n_tokens, out_token_stride, per, out_id_stride, D) * dtype_bytes(out_dtype);
  if (overlap(out, ob, ids, extent(n_tokens, ids_stride, 1, 0, n_ids) * 4) ||
      overlap(out, ob, table, extent(rows, table_stride, 1, 0, D) * dtype_bytes(table_dtype)) ||
      overlap(out, ob, status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out overlaps an input", fn);
  if ((st = engram::check_sm103()) != ENGRAM_OK) return st;
  engram::EmbedParams p{};
  p.ids = ids;
  p.table = table;
  p.out = out;
  p.status = status;
  p.n_tokens = n_tokens;
  p.ids_stride = ids_stride;
  p.rows = rows;
  p.table_stride = table_stride;
  p.out_token_stride = out_token_stride;
  p.out_id_stride = out_id_stride;
  p.n_ids = n_ids;
  p.D = D;
  p.scale = scale;
  return launched("engram_embed launch", engram::launch_embed(p, table_dtype, out_dtype, pooled != 0,
                                                              (cudaStream_t)stream));
}

ENGRAM_API size_t engram_embed_grad_workspace_bytes(int64_t n_tokens, int32_t n_ids, int32_t D) {
  if (n_tokens < 0 || n_ids < 1 || n_tokens > INT32_MAX / n_ids || D < 1 || D > ENGRAM_MAX_EMBED_D)
    return 0;
  return engram::embed_grad_workspace_bytes(n_tokens * n_ids, D);
}

// The checks and the launch that the two gradient calls share; `out_rows` rows of grad.
static engram_status embed_grad_common(const char *fn, const int32_t *ids, int64_t n_tokens,
                                       int32_t n_ids, int64_t ids_stride, const void *dy,
                                       int32_t dy_dtype, int64_t dy_token_stride,
                                       int64_t dy_id_stride, int64_t rows, int32_t D, float scale,
                                       bool accumulate, void *grad, int32_t grad_dtype,
                                       int64_t grad_stride, bool sparse, int32_t *row_ids_out,
                                       int32_t *count_out, void *workspace,
                                       size_t workspace_bytes, int32_t *status, void *stream) {
  engram_status st = check_ids(fn, ids, n_tokens, n_ids, ids_stride, rows, D, status);
  if (st != ENGRAM_OK) return st;
  if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  const int64_t n = n_tokens * n_ids, out_rows = sparse ? n : rows;
  if (dy_id_stride < 0 || dy_token_stride < 0)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: dy strides < 0", fn);
  if (n > 0 && (!dy || !aligned(dy, dtype_bytes(dy_dtype))))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: dy NULL or misaligned", fn);
  if ((out_rows > 0 && (!grad || !aligned(grad, dtype_bytes(grad_dtype)))) ||
      (out_rows > 1 && grad_stride < D))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: gradient NULL or misaligned, or its stride under D", fn);
  if (sparse && (!count_out || !aligned(count_out, 4) || (n > 0 && !row_ids_out) ||
                 !aligned(row_ids_out, 4)))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: row_ids_out or count_out NULL or misaligned", fn);
  const size_t need = engram_embed_grad_workspace_bytes(n_tokens, n_ids, D);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: workspace NULL, not 16-byte aligned or under %zu bytes", fn, need);
  const struct {
    const void *p;
    size_t n;
  } outs[4] = {{grad, extent(out_rows, grad_stride, 1, 0, D) * dtype_bytes(grad_dtype)},
               {workspace, need},
               {sparse ? row_ids_out : nullptr, (size_t)n * 4},
               {sparse ? count_out : nullptr, 4}},
    ins[3] = {{ids, (size_t)extent(n_tokens, ids_stride, 1, 0, n_ids) * 4},
              {dy, extent(n_tokens, dy_token_stride, n_ids, dy_id_stride, D) * dtype_bytes(dy_dtype)},
              {status, 4}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i)
      if (overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o].p, outs[o].n, outs[i].p, outs[i].n))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  if ((st = engram::check_sm103()) != ENGRAM_OK) return st;
  engram::EmbedGradParams p{};
  p.ids = ids;
  p.dy = dy;
  p.grad = grad;
  p.row_ids_out = row_ids_out;
  p.count_out = count_out;
  p.status = status;
  p.n = n;
  p.ids_stride = ids_stride;
  p.rows = rows;
  p.dy_token_stride = dy_token_stride;
  p.dy_id_stride = dy_id_stride;
  p.grad_stride = grad_stride;
  p.n_ids = n_ids;
  p.D = D;
  p.scale = scale;
  p.accumulate = accumulate;
  return launched(fn, engram::launch_embed_grad(p, dy_dtype, grad_dtype, workspace, sparse,
                                                (cudaStream_t)stream));
}

ENGRAM_API engram_status engram_embed_grad(const int32_t *ids, int64_t n_tokens, int32_t n_ids,
                                           int64_t ids_stride, const void *dy, int32_t dy_dtype,
                                           int64_t dy_token_stride, int64_t dy_id_stride,
                                           int64_t rows, int32_t D, float scale,
                                           int32_t accumulate, void *grad, int32_t grad_dtype,
                                           int64_t grad_stride, void *workspace,
                                           size_t workspace_bytes, int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_embed_grad");
  return embed_grad_common("engram_embed_grad", ids, n_tokens, n_ids, ids_stride, dy, dy_dtype,
                           dy_token_stride, dy_id_stride, rows, D, scale, accumulate != 0, grad,
                           grad_dtype, grad_stride, false, nullptr, nullptr, workspace,
                           workspace_bytes, status, stream);
}

ENGRAM_API engram_status engram_embed_grad_rows(const int32_t *ids, int64_t n_tokens, int32_t n_ids,
                                                int64_t ids_stride, const void *dy,
                                                int32_t dy_dtype, int64_t dy_token_stride,
                                                int64_t dy_id_stride, int64_t rows, int32_t D,
                                                float scale, int32_t *row_ids_out, void *grads_out,
                                                int32_t grads_dtype, int64_t grads_stride,
                                                int32_t *count_out, void *workspace,
                                                size_t workspace_bytes, int32_t *status,
                                                void *stream) {
  ENGRAM_NVTX_RANGE("engram_embed_grad_rows");
  return embed_grad_common("engram_embed_grad_rows", ids, n_tokens, n_ids, ids_stride, dy, dy_dtype,
                           dy_token_stride, dy_id_stride, rows, D, scale, false, grads_out,
                           grads_dtype, grads_stride, true, row_ids_out, count_out, workspace,
                           workspace_bytes, status, stream);
}

ENGRAM_API engram_status engram_fp8_quantise(const void *x, int32_t x_dtype, int64_t M, int64_t K,
                                             int64_t x_stride, int32_t block_rows, uint8_t *q,
                                             int64_t q_stride, uint8_t *s, uint8_t *qt,
                                             int64_t qt_stride, uint8_t *st, int32_t *status,
                                             void *stream) {
  ENGRAM_NVTX_RANGE("engram_fp8_quantise");
  const char *fn = "engram_fp8_quantise";
  if (M < 0 || K < 1 || M > INT32_MAX || K > INT32_MAX)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: M in [0, 2^31-1] and K in [1, 2^31-1]", fn);
  const int64_t kb = (K + 127) / 128, mb = (M + 127) / 128;
  if (mb * kb > INT32_MAX - 4096 || M * kb / 16 > INT32_MAX)
    return set_error(ENGRAM_ERR_UNSUPPORTED, "%s: over 2^31-1 tiles", fn);
  if (!dtype_ok(x_dtype)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown x dtype", fn);
  if (block_rows != 1 && block_rows != ENGRAM_FP8_BLOCK)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: block_rows must be 1 or %d", fn, ENGRAM_FP8_BLOCK);
  if (M == 0) return ok();  // empty buffers have no address
  if ((!q && !qt) || (q && !s) || (qt && !st))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: q or qt must be given, each with its scales", fn);
  if (!aligned(status, 4)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: status misaligned", fn);
  if (!x || !aligned(x, dtype_bytes(x_dtype)) || (M > 1 && x_stride < K))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: x NULL or misaligned, or its stride under K", fn);
  if (!aligned(q, 16) || !aligned(qt, 16) || (q && M > 1 && (q_stride < K || q_stride % 16 != 0)) ||
      (qt && K > 1 && (qt_stride < M || qt_stride % 16 != 0)))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: q and qt must be 16-byte aligned, their strides multiples of 16 that hold a row",
                     fn);
  const size_t xb = extent(M, x_stride, 1, 0, K) * dtype_bytes(x_dtype);
  const size_t sn = (block_rows == 1 ? M : mb) * kb, tn = (block_rows == 1 ? K : kb) * mb;
  const struct {
    const void *p;
    size_t n;
  } outs[4] = {{q, q ? (size_t)extent(M, q_stride, 1, 0, K) : 0}, {q ? s : nullptr, sn},
               {qt, qt ? (size_t)extent(K, qt_stride, 1, 0, M) : 0}, {qt ? st : nullptr, tn}};
  for (int o = 0; o < 4; ++o) {
    if (overlap(outs[o].p, outs[o].n, x, xb) || overlap(outs[o].p, outs[o].n, status, 4))
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps x or status", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o].p, outs[o].n, outs[i].p, outs[i].n))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  engram_status code = engram::check_sm103();
  if (code != ENGRAM_OK) return code;
  engram::QuantiseParams p{};
  p.x = x;
  p.q = q;
  p.s = s;
  p.qt = qt;
  p.st = st;
  p.status = status;
  p.wait_limit_ns = engram::wait_limit_ns();
  p.M = M;
  p.K = K;
  p.x_stride = x_stride;
  p.q_stride = q_stride;
  p.qt_stride = qt_stride;
  p.block_rows = block_rows;
  return launched("engram_fp8_quantise launch",
                  engram::launch_quantise(p, x_dtype, (cudaStream_t)stream));
}

ENGRAM_API engram_status engram_fp8_matmul(const uint8_t *a, int64_t a_stride, const uint8_t *a_scale,
                                           int32_t a_block, const uint8_t *b, int64_t b_stride,
                                           const uint8_t *b_scale, int32_t b_block, int64_t M,
                                           int64_t N, int64_t K, void *out, int32_t out_dtype,
                                           int64_t out_stride, int32_t *status, void *stream) {
  ENGRAM_NVTX_RANGE("engram_fp8_matmul");
  const char *fn = "engram_fp8_matmul";
  const int64_t most = INT32_MAX - 256;  // tile origins stay in 32 bits
  if (M < 0 || N < 0 || K < 1 || M > most || N > most || K > most)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: M, N >= 0 and K >= 1, all under 2^31 - 256", fn);
  if ((a_block != 1 && a_block != ENGRAM_FP8_BLOCK) || (b_block != 1 && b_block != ENGRAM_FP8_BLOCK))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: a_block and b_block must be 1 or %d", fn,
                     ENGRAM_FP8_BLOCK);
  if (!dtype_ok(out_dtype)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown out dtype", fn);
  if (M == 0 || N == 0) return ok();
  if (!a || !a_scale || !b || !b_scale || !out)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: NULL buffer", fn);
  // One row needs no stride, but the copies' descriptors take one all the same.
  const int64_t one = (K + 15) / 16 * 16;
  if (M == 1) a_stride = one;
  if (N == 1) b_stride = one;
  if (!aligned(a, 16) || !aligned(b, 16) || a_stride < K || b_stride < K || a_stride % 16 != 0 ||
      b_stride % 16 != 0)
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: a and b must be 16-byte aligned, their strides multiples of 16 from K on", fn);
  if (!aligned(out, dtype_bytes(out_dtype)) || (M > 1 && out_stride < N) || !aligned(status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out misaligned or its stride under N", fn);
  const int64_t kb = (K + 127) / 128;
  const size_t ob = extent(M, out_stride, 1, 0, N) * dtype_bytes(out_dtype);
  if (overlap(out, ob, a, extent(M, a_stride, 1, 0, K)) ||
      overlap(out, ob, b, extent(N, b_stride, 1, 0, K)) ||
      overlap(out, ob, a_scale, ((M - 1) / a_block + 1) * kb) ||
      overlap(out, ob, b_scale, ((N - 1) / b_block + 1) * kb) || overlap(out, ob, status, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: out overlaps an input", fn);
  engram_status st = engram::check_sm103();
  if (st != ENGRAM_OK) return st;
  engram::MatmulParams p{};
  p.a = a;
  p.a_scale = a_scale;
  p.b = b;
  p.b_scale = b_scale;
  p.out = out;
  p.status = status;
  p.M = M;
  p.N = N;
  p.K = K;
  p.a_stride = a_stride;
  p.b_stride = b_stride;
  p.out_stride = out_stride;
  p.a_block = a_block;
  p.b_block = b_block;
  return launched("engram_fp8_matmul launch",
                  engram::launch_fp8_matmul(p, out_dtype, (cudaStream_t)stream));
}

ENGRAM_API size_t engram_gate_add_grad_workspace_bytes(void) {
  return engram::kGateGradMaxBlocks * sizeof(float4);
}

ENGRAM_API engram_status engram_gate_add_grad(const float *k, const uint8_t *state,
                                              int64_t n_tokens, int32_t D,
                                              const uint16_t *streams_in, const float *alpha,
                                              float eps, const uint16_t *dy, uint16_t *dx,
                                              void *dk, int32_t dk_dtype, float *dalpha,
                                              void *workspace, size_t workspace_bytes,
                                              void *stream) {
  ENGRAM_NVTX_RANGE("engram_gate_add_grad");
  const char *fn = "engram_gate_add_grad";
  if (n_tokens < 0 || n_tokens > INT32_MAX)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: n_tokens out of range", fn);
  if (D < 16 || D % 16 != 0 || D > 8192)
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: D must be a multiple of 16 in [16, 8192]", fn);
  if (!dtype_ok(dk_dtype)) return set_error(ENGRAM_ERR_INVALID_ARG, "%s: unknown dk dtype", fn);
  if (!alpha || !dalpha || !aligned(alpha, 4) || !aligned(dalpha, 4))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: alpha or dalpha NULL or misaligned", fn);
  if (!(eps >= 0.f) || !isfinite(eps))
    return set_error(ENGRAM_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  const size_t need = engram_gate_add_grad_workspace_bytes();
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return set_error(ENGRAM_ERR_INVALID_ARG,
                     "%s: workspace NULL, not 16-byte aligned or under %zu bytes", fn, need);
  const size_t sb = (size_t)n_tokens * 4 * D * 2, kb = (size_t)n_tokens * D * 4;
  const size_t db = (size_t)n_tokens * D * dtype_bytes(dk_dtype);
  if (n_tokens > 0) {
    if (!k || !streams_in || !dy || !dx || !dk)
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: NULL buffer", fn);
    if (!aligned(k, 16) || !aligned(streams_in, 16) || !aligned(dy, 16) || !aligned(dx, 16) ||
        !aligned(dk, 16))
      return set_error(ENGRAM_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  }
  const struct {
    const void *p;
    size_t n;
  } outs[4] = {{dx, sb}, {dk, db}, {dalpha, 16}, {workspace, need}},
    ins[5] = {{k, kb}, {state, state ? (size_t)n_tokens : 0}, {streams_in, sb}, {alpha, 16}, {dy, sb}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (!(o == 0 && i == 4 && dx == dy) && overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o].p, outs[o].n, outs[i].p, outs[i].n))
        return set_error(ENGRAM_ERR_INVALID_ARG, "%s: output buffers overlap", fn);
  }
  engram_status st = engram::check_sm103();
  if (st != ENGRAM_OK) return st;
  engram::GateGradParams p{};
  p.k = k;
  p.state = state;
  p.x = streams_in;
  p.dy = dy;
  p.dx = dx;
  p.dk = dk;
  p.alpha = alpha;
  p.partial = static_cast<float4 *>(workspace);
  p.dalpha = dalpha;
  p.T = n_tokens;
  p.D = D;
  p.eps = eps;
  return launched("engram_gate_add_grad launch",
                  engram::launch_gate_grad(p, dk_dtype, (cudaStream_t)stream));
}

}  // extern "C"

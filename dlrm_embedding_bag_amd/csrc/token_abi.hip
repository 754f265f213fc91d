// token_abi.hip -- the extern "C" entry points of the token operators:
// argument validation only.  Every argument error is reported before any work
// is enqueued; nothing here allocates memory, throws or synchronizes.
#include <limits.h>
#include <math.h>

#include "../../include/dlrm_embedding_bag.h"
#include "kernels.hpp"

using namespace dlrm;

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? DLRM_OK : DLRM_ERR_HIP; }

bool float_dtype(int32_t t) { return t == DLRM_F32 || t == DLRM_BF16; }

// Row stride of an input (0 repeats one row) and of an output.
bool in_stride(int64_t ld, int64_t cols) { return ld == 0 || ld >= cols; }
bool out_stride(int64_t ld, int64_t cols) { return ld >= cols; }

// The largest |product sum| of k int8 pairs, 128 * 128 * k, stays below 2^31.
constexpr int32_t kMaxI8K = 131071;
constexpr int32_t kMaxI8Rows = 1 << 26;  // of either operand: a launch holds < 2^32 threads

bool lookup_shape(int64_t n, int64_t rows, int32_t dim) {
  return n >= 0 && n <= INT32_MAX && rows >= 1 && rows < INT32_MAX && dim >= 1 &&
         dim <= DLRM_MAX_TOKEN_DIM;
}

}  // namespace

extern "C" {

int emb_lookup_scaled(int64_t num_tokens, int64_t rows, int32_t dim, const void *table,
                      int64_t ld_table, int32_t table_dtype, const int32_t *tokens, float scale,
                      void *out, int64_t ld_out, int32_t out_dtype, void *stream) {
  if (!lookup_shape(num_tokens, rows, dim)) return DLRM_ERR_SHAPE;
  if (!float_dtype(table_dtype) && table_dtype != DLRM_FP8_E4M3) return DLRM_ERR_SHAPE;
  if (!float_dtype(out_dtype)) return DLRM_ERR_SHAPE;
  if (!in_stride(ld_table, dim) || !out_stride(ld_out, dim)) return DLRM_ERR_SHAPE;
  if (num_tokens == 0) return DLRM_OK;
  if (!table || !tokens || !out) return DLRM_ERR_NULL;
  LookupParams p{};
  p.tokens = num_tokens;
  p.rows = rows;
  p.dim = dim;
  p.table = table;
  p.ld_table = ld_table;
  p.token = tokens;
  p.scale = scale;
  p.out = out;
  p.ld_out = ld_out;
  return status_of(launch_lookup(p, table_dtype, out_dtype, (hipStream_t)stream));
}

size_t emb_lookup_grad_workspace_bytes(int64_t num_tokens, int64_t rows, int32_t dim) {
  return lookup_shape(num_tokens, rows, dim) ? lookup_grad_workspace(num_tokens, rows, dim) : 0;
}

int emb_lookup_grad(int64_t num_tokens, int64_t rows, int32_t dim, const void *grad,
                    int64_t ld_grad, int32_t grad_dtype, const int32_t *tokens, float scale,
                    int32_t accumulate, void *out, int64_t ld_out, int32_t out_dtype,
                    void *workspace, size_t workspace_bytes, void *stream) {
  if (!lookup_shape(num_tokens, rows, dim)) return DLRM_ERR_SHAPE;
  if (!float_dtype(grad_dtype) || !float_dtype(out_dtype)) return DLRM_ERR_SHAPE;
  if (!in_stride(ld_grad, dim) || !out_stride(ld_out, dim)) return DLRM_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return DLRM_ERR_SHAPE;
  if (num_tokens == 0 && accumulate) return DLRM_OK;
  if (!out || (num_tokens > 0 && (!grad || !tokens))) return DLRM_ERR_NULL;
  const size_t need = lookup_grad_workspace(num_tokens, rows, dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DLRM_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return DLRM_ERR_WORKSPACE;
  GradParams p{};
  p.n = num_tokens;
  p.rows = rows;
  p.dim = dim;
  p.grad = grad;
  p.ld_grad = ld_grad;
  p.token = tokens;
  p.scale = scale;
  p.out = out;
  p.ld_out = ld_out;
  p.accumulate = accumulate;
  return status_of(launch_lookup_grad(p, grad_dtype, out_dtype, workspace, (hipStream_t)stream));
}

int rms_norm_residual_i8(int64_t m, int32_t dim, const void *x, int64_t ldx, const void *residual,
                         int64_t ldr, int32_t dtype, const float *weight, double eps, void *h,
                         int64_t ldh, int8_t *codes, int64_t ldq, float *scale, void *stream) {
  if (m < 0 || dim < 1 || dim > DLRM_MAX_TOKEN_DIM || !float_dtype(dtype)) return DLRM_ERR_SHAPE;
  if (!(eps >= 0.0) || !(eps < INFINITY)) return DLRM_ERR_SHAPE;
  if (!in_stride(ldx, dim) || !out_stride(ldq, dim)) return DLRM_ERR_SHAPE;
  if (residual && (!in_stride(ldr, dim) || !out_stride(ldh, dim))) return DLRM_ERR_SHAPE;
  if (m == 0) return DLRM_OK;
  if (!x || !codes || !scale || (residual && !h)) return DLRM_ERR_NULL;
  NormParams p{};
  p.m = m;
  p.dim = dim;
  p.x = x;
  p.ldx = ldx;
  p.residual = residual;
  p.ldr = ldr;
  p.weight = weight;
  p.eps = eps;
  p.h = h;
  p.ldh = ldh;
  p.codes = codes;
  p.ldq = ldq;
  p.scale = scale;
  return status_of(launch_rms_norm_i8(p, dtype, (hipStream_t)stream));
}

int linear_i8_bias_act(int32_t m, int32_t n, int32_t k, const int8_t *a, int64_t lda,
                       const float *a_scale, const int8_t *w, int64_t ldw, const float *w_scale,
                       const float *bias, int32_t act, void *c, int64_t ldc, int32_t out_dtype,
                       void *stream) {
  if (m < 0 || n < 1 || k < 1) return DLRM_ERR_SHAPE;
  if (act != DLRM_ACT_NONE && act != DLRM_ACT_RELU && act != DLRM_ACT_SIGMOID)
    return DLRM_ERR_SHAPE;
  if (!float_dtype(out_dtype)) return DLRM_ERR_SHAPE;
  if (!in_stride(lda, k) || !out_stride(ldw, k) || !out_stride(ldc, n)) return DLRM_ERR_SHAPE;
  if (k > kMaxI8K || m > kMaxI8Rows || n > kMaxI8Rows) return DLRM_ERR_UNSUPPORTED;
  if (m == 0) return DLRM_OK;
  if (!a || !a_scale || !w || !w_scale || !c) return DLRM_ERR_NULL;
  LinearI8Params p{};
  p.M = m;
  p.N = n;
  p.K = k;
  p.A = a;
  p.lda = lda;
  p.a_scale = a_scale;
  p.W = w;
  p.ldw = ldw;
  p.w_scale = w_scale;
  p.bias = bias;
  p.act = act;
  p.C = c;
  p.ldc = ldc;
  return status_of(launch_linear_i8(p, out_dtype, (hipStream_t)stream));
}

}  // extern "C"

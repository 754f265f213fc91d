// attention_abi.hip -- the extern "C" entry points of the attention operators:
// argument validation only.  Every argument error is reported before any work
// is enqueued; nothing here allocates memory, throws or synchronizes.
#include <limits.h>
#include <math.h>

#include <initializer_list>

#include "../../include/dlrm_embedding_bag.h"
#include "kernels.hpp"

using namespace dlrm;

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? DLRM_OK : DLRM_ERR_HIP; }

bool float_dtype(int32_t t) { return t == DLRM_F32 || t == DLRM_BF16; }
int size_of(int32_t dtype) { return dtype == DLRM_F32 ? 4 : 2; }

// (n, heads, dim) rows of an input may repeat; an output's must not overlap, in
// either order of its outer dimensions.
bool in_rows(int64_t token, int64_t head) { return token >= 0 && head >= 0; }
bool out_rows(int64_t n, int32_t heads, int32_t dim, int64_t token, int64_t head) {
  if (n <= 0 || heads <= 0) return true;
  const __int128 t = token, h = head;
  const bool token_outer =
      (heads == 1 || h >= dim) && (n == 1 || t >= (__int128)(heads - 1) * h + dim);
  const bool head_outer =
      (n == 1 || t >= dim) && (heads == 1 || h >= (__int128)(n - 1) * t + dim);
  return token >= 0 && head >= 0 && (token_outer || head_outer);
}

constexpr int32_t kMaxHeads = 1 << 16;

bool rope_shape(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim, int32_t pairs,
                int32_t dtype) {
  return tokens >= 0 && tokens <= INT32_MAX && heads >= 0 && heads <= kMaxHeads && kv_heads >= 0 &&
         kv_heads <= kMaxHeads && heads + kv_heads >= 1 && dim >= 8 && dim <= DLRM_MAX_ROPE_DIM &&
         dim % 8 == 0 && pairs >= 4 && pairs % 4 == 0 && 2 * pairs <= dim && float_dtype(dtype);
}

// 16-byte accesses: the address and every stride that is walked.
bool aligned_rows(const void *p, int64_t n, int64_t token, int32_t heads, int64_t head,
                  int32_t dtype) {
  const int64_t e = 16 / size_of(dtype);
  return aligned16(p) && (n <= 1 || token % e == 0) && (heads <= 1 || head % e == 0);
}
// The kernels keep scores in units of log 2, so that factor has to be a number too.
bool scale_of_scores(float scale) { return scale > 0.0f && scale * kLog2e < INFINITY; }

// Tiles of up to 128 rows are addressed within 2 GiB.
constexpr int64_t kMaxTokenStride = (1 << 22) - 1024;
bool near_rows(int64_t n, std::initializer_list<int64_t> strides) {
  for (const int64_t s : strides)
    if (n > 1 && s > kMaxTokenStride) return false;
  return true;
}

int attention_shape(int64_t tokens, int64_t kv_tokens, int64_t batch, int32_t heads,
                    int32_t kv_heads, int32_t dim, int32_t dtype, int32_t causal, float scale) {
  if (tokens < 0 || tokens > INT32_MAX || kv_tokens < 0 || kv_tokens > INT32_MAX || batch < 1 ||
      batch >= INT32_MAX || heads < 1 || heads > kMaxHeads || kv_heads < 1 || kv_heads > heads ||
      heads % kv_heads || dim < 8 || dim % 8 || !float_dtype(dtype) ||
      (causal != 0 && causal != 1) || !scale_of_scores(scale))
    return DLRM_ERR_SHAPE;
  return dim > DLRM_MAX_ATTENTION_DIM ? DLRM_ERR_UNSUPPORTED : DLRM_OK;
}

// DLRM_ERR_UNSUPPORTED only for what a cache could hold and this one does not.
int cache_shape(int32_t heads, int32_t dim, int64_t pages, int32_t page, int32_t bits) {
  if (heads < 1 || heads > kMaxHeads || pages < 1 || dim < 1 || page < 1) return DLRM_ERR_SHAPE;
  if ((bits != 4 && bits != 8) || (dim != 32 && dim != 64 && dim != 128) || page < 16 ||
      page > DLRM_MAX_CACHE_PAGE || (page & (page - 1)))
    return DLRM_ERR_UNSUPPORTED;
  return pages * (__int128)page > INT32_MAX ? DLRM_ERR_SHAPE : DLRM_OK;
}

}  // namespace

extern "C" {

int qk_norm_rope(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                 const void *q, int64_t q_token, int64_t q_head, const void *k, int64_t k_token,
                 int64_t k_head, const int32_t *positions, const float *freqs, int32_t pairs,
                 int32_t interleaved, const float *q_weight, const float *k_weight, double eps,
                 void *out_q, int64_t oq_token, int64_t oq_head, void *out_k, int64_t ok_token,
                 int64_t ok_head, void *stream) {
  if (!rope_shape(tokens, heads, kv_heads, dim, pairs, dtype)) return DLRM_ERR_SHAPE;
  if (interleaved != 0 && interleaved != 1) return DLRM_ERR_SHAPE;
  if (!(eps >= 0.0) || !(eps < INFINITY)) return DLRM_ERR_SHAPE;
  if (!in_rows(q_token, q_head) || !in_rows(k_token, k_head)) return DLRM_ERR_SHAPE;
  if (!out_rows(tokens, heads, dim, oq_token, oq_head) ||
      !out_rows(tokens, kv_heads, dim, ok_token, ok_head))
    return DLRM_ERR_SHAPE;
  if (tokens == 0) return DLRM_OK;
  if (!positions || !freqs || (heads && (!q || !out_q)) || (kv_heads && (!k || !out_k)))
    return DLRM_ERR_NULL;
  RopeParams p{};
  p.tokens = tokens;
  p.dim = dim;
  p.pairs = pairs;
  p.positions = positions;
  p.freqs = freqs;
  p.eps = eps;
  p.q = {heads, q, q_token, q_head, q_weight, out_q, oq_token, oq_head, nullptr, 0, 0, nullptr};
  p.k = {kv_heads, k, k_token, k_head, k_weight, out_k, ok_token, ok_head, nullptr, 0, 0, nullptr};
  return status_of(launch_rope(p, dtype, interleaved != 0, (hipStream_t)stream));
}

size_t qk_norm_rope_grad_workspace_bytes(int64_t tokens, int32_t dim) {
  return tokens >= 0 && tokens <= INT32_MAX && dim >= 8 && dim <= DLRM_MAX_ROPE_DIM
             ? rope_grad_workspace(tokens, dim)
             : 0;
}

int qk_norm_rope_grad(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                      const void *grad_q, int64_t gq_token, int64_t gq_head, const void *grad_k,
                      int64_t gk_token, int64_t gk_head, const void *q, int64_t q_token,
                      int64_t q_head, const void *k, int64_t k_token, int64_t k_head,
                      const int32_t *positions, const float *freqs, int32_t pairs,
                      int32_t interleaved, const float *q_weight, const float *k_weight,
                      double eps, void *out_q, int64_t oq_token, int64_t oq_head, void *out_k,
                      int64_t ok_token, int64_t ok_head, float *out_q_weight, float *out_k_weight,
                      void *workspace, size_t workspace_bytes, void *stream) {
  if (!rope_shape(tokens, heads, kv_heads, dim, pairs, dtype)) return DLRM_ERR_SHAPE;
  if (interleaved != 0 && interleaved != 1) return DLRM_ERR_SHAPE;
  if (!(eps >= 0.0) || !(eps < INFINITY)) return DLRM_ERR_SHAPE;
  if (!in_rows(q_token, q_head) || !in_rows(k_token, k_head) || !in_rows(gq_token, gq_head) ||
      !in_rows(gk_token, gk_head))
    return DLRM_ERR_SHAPE;
  if (!out_rows(tokens, heads, dim, oq_token, oq_head) ||
      !out_rows(tokens, kv_heads, dim, ok_token, ok_head))
    return DLRM_ERR_SHAPE;
  const bool weights = out_q_weight || out_k_weight;
  if (tokens == 0 && !weights) return DLRM_OK;
  if (tokens > 0 &&
      (!positions || !freqs || (heads && (!q || !grad_q || !out_q)) ||
       (kv_heads && (!k || !grad_k || !out_k))))
    return DLRM_ERR_NULL;
  const size_t need = weights ? rope_grad_workspace(tokens, dim) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return DLRM_ERR_WORKSPACE;
  RopeParams p{};
  p.tokens = tokens;
  p.dim = dim;
  p.pairs = pairs;
  p.positions = positions;
  p.freqs = freqs;
  p.eps = eps;
  p.q = {heads,   q,        q_token, q_head,   q_weight, out_q,
         oq_token, oq_head, grad_q,  gq_token, gq_head,  out_q_weight};
  p.k = {kv_heads, k,       k_token, k_head,   k_weight, out_k,
         ok_token, ok_head, grad_k,  gk_token, gk_head,  out_k_weight};
  return status_of(launch_rope_grad(p, dtype, interleaved != 0, workspace, (hipStream_t)stream));
}

int attention_packed(int64_t tokens, int64_t kv_tokens, int64_t batch, int32_t heads,
                     int32_t kv_heads, int32_t dim, int32_t dtype, const void *q, int64_t q_token,
                     int64_t q_head, const void *k, int64_t k_token, int64_t k_head, const void *v,
                     int64_t v_token, int64_t v_head, const int32_t *offsets,
                     const int32_t *kv_offsets, int32_t causal, float scale, int32_t fill,
                     void *out, int64_t o_token, int64_t o_head, float *lse, void *stream) {
  const int bad =
      attention_shape(tokens, kv_tokens, batch, heads, kv_heads, dim, dtype, causal, scale);
  if (bad) return bad;
  if (fill < 0 || fill > 3 || (!kv_offsets && kv_tokens != tokens)) return DLRM_ERR_SHAPE;
  if (!in_rows(q_token, q_head) || !in_rows(k_token, k_head) || !in_rows(v_token, v_head))
    return DLRM_ERR_SHAPE;
  if (!out_rows(tokens, heads, dim, o_token, o_head)) return DLRM_ERR_SHAPE;
  if (tokens == 0) return DLRM_OK;
  if (!offsets || !q || !out || (kv_tokens > 0 && (!k || !v))) return DLRM_ERR_NULL;
  if (!aligned_rows(q, tokens, q_token, heads, q_head, dtype) ||
      !aligned_rows(k, kv_tokens, k_token, kv_heads, k_head, dtype) ||
      !aligned_rows(v, kv_tokens, v_token, kv_heads, v_head, dtype) ||
      !aligned_rows(out, tokens, o_token, heads, o_head, dtype))
    return DLRM_ERR_UNSUPPORTED;
  if (!near_rows(tokens, {q_token, o_token}) || !near_rows(kv_tokens, {k_token, v_token}))
    return DLRM_ERR_UNSUPPORTED;
  AttentionParams p{};
  p.tokens = tokens;
  p.kv_tokens = kv_tokens;
  p.batch = batch;
  p.heads = heads;
  p.group = heads / kv_heads;
  p.dim = dim;
  p.q = {q, tokens > 1 ? q_token : dim, q_head};
  p.k = {k, kv_tokens > 1 ? k_token : dim, k_head};
  p.v = {v, kv_tokens > 1 ? v_token : dim, v_head};
  p.offsets = offsets;
  p.kv_offsets = kv_offsets;
  p.causal = causal;
  p.scale = scale;
  p.fill = lse ? fill : fill & 1;
  p.out = {out, tokens > 1 ? o_token : dim, o_head};
  p.lse = lse;
  return status_of(launch_attention(p, dtype, (hipStream_t)stream));
}

size_t attention_packed_grad_workspace_bytes(int64_t tokens, int32_t heads) {
  return tokens >= 0 && tokens <= INT32_MAX && heads >= 1 && heads <= kMaxHeads
             ? attention_grad_workspace(tokens, heads)
             : 0;
}

int attention_packed_grad(int64_t tokens, int64_t kv_tokens, int64_t batch, int32_t heads,
                          int32_t kv_heads, int32_t dim, int32_t dtype, const void *grad,
                          int64_t g_token, int64_t g_head, const void *q, int64_t q_token,
                          int64_t q_head, const void *k, int64_t k_token, int64_t k_head,
                          const void *v, int64_t v_token, int64_t v_head, const void *out,
                          int64_t o_token, int64_t o_head, const float *lse,
                          const int32_t *offsets, const int32_t *kv_offsets, int32_t causal,
                          float scale, int32_t fill, void *dq, int64_t dq_token, int64_t dq_head,
                          void *dk, int64_t dk_token, int64_t dk_head, void *dv, int64_t dv_token,
                          int64_t dv_head, void *workspace, size_t workspace_bytes, void *stream) {
  const int bad =
      attention_shape(tokens, kv_tokens, batch, heads, kv_heads, dim, dtype, causal, scale);
  if (bad) return bad;
  if (fill < 0 || fill > 7 || (!kv_offsets && kv_tokens != tokens)) return DLRM_ERR_SHAPE;
  if (!in_rows(g_token, g_head) || !in_rows(q_token, q_head) || !in_rows(k_token, k_head) ||
      !in_rows(v_token, v_head) || !in_rows(o_token, o_head))
    return DLRM_ERR_SHAPE;
  if (!out_rows(tokens, heads, dim, dq_token, dq_head) ||
      !out_rows(kv_tokens, kv_heads, dim, dk_token, dk_head) ||
      !out_rows(kv_tokens, kv_heads, dim, dv_token, dv_head))
    return DLRM_ERR_SHAPE;
  if (tokens == 0 && kv_tokens == 0) return DLRM_OK;
  if (!offsets || (tokens > 0 && (!grad || !q || !out || !lse || !dq)) ||
      (kv_tokens > 0 && (!k || !v || !dk || !dv)))
    return DLRM_ERR_NULL;
  if (!aligned_rows(grad, tokens, g_token, heads, g_head, dtype) ||
      !aligned_rows(q, tokens, q_token, heads, q_head, dtype) ||
      !aligned_rows(k, kv_tokens, k_token, kv_heads, k_head, dtype) ||
      !aligned_rows(v, kv_tokens, v_token, kv_heads, v_head, dtype) ||
      !aligned_rows(out, tokens, o_token, heads, o_head, dtype) ||
      !aligned_rows(dq, tokens, dq_token, heads, dq_head, dtype) ||
      !aligned_rows(dk, kv_tokens, dk_token, kv_heads, dk_head, dtype) ||
      !aligned_rows(dv, kv_tokens, dv_token, kv_heads, dv_head, dtype))
    return DLRM_ERR_UNSUPPORTED;
  if (!near_rows(tokens, {q_token, g_token, o_token, dq_token}) ||
      !near_rows(kv_tokens, {k_token, v_token, dk_token, dv_token}))
    return DLRM_ERR_UNSUPPORTED;
  const size_t need = attention_grad_workspace(tokens, heads);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return DLRM_ERR_WORKSPACE;
  AttentionGradParams p{};
  p.tokens = tokens;
  p.kv_tokens = kv_tokens;
  p.batch = batch;
  p.heads = heads;
  p.group = heads / kv_heads;
  p.dim = dim;
  p.grad = {grad, tokens > 1 ? g_token : dim, g_head};
  p.q = {q, tokens > 1 ? q_token : dim, q_head};
  p.k = {k, kv_tokens > 1 ? k_token : dim, k_head};
  p.v = {v, kv_tokens > 1 ? v_token : dim, v_head};
  p.out = {out, tokens > 1 ? o_token : dim, o_head};
  p.lse = lse;
  p.offsets = offsets;
  p.kv_offsets = kv_offsets;
  p.causal = causal;
  p.scale = scale;
  p.fill = fill;
  p.dq = {dq, tokens > 1 ? dq_token : dim, dq_head};
  p.dk = {dk, kv_tokens > 1 ? dk_token : dim, dk_head};
  p.dv = {dv, kv_tokens > 1 ? dv_token : dim, dv_head};
  return status_of(launch_attention_grad(p, dtype, workspace, (hipStream_t)stream));
}

int kv_cache_write(int64_t tokens, int32_t heads, int32_t dim, int32_t dtype, const void *k,
                   int64_t k_token, int64_t k_head, const void *v, int64_t v_token, int64_t v_head,
                   const int32_t *slots, int64_t pages, int32_t page, int32_t bits, void *k_codes,
                   void *k_scales, void *v_codes, void *v_scales, void *stream) {
  if (tokens < 0 || tokens > INT32_MAX || !float_dtype(dtype)) return DLRM_ERR_SHAPE;
  const int bad = cache_shape(heads, dim, pages, page, bits);
  if (bad) return bad;
  if (!in_rows(k_token, k_head) || !in_rows(v_token, v_head)) return DLRM_ERR_SHAPE;
  if (tokens == 0) return DLRM_OK;
  if (!k || !v || !slots || !k_codes || !k_scales || !v_codes || !v_scales) return DLRM_ERR_NULL;
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_scales) || !aligned16(v_scales))
    return DLRM_ERR_UNSUPPORTED;
  CacheParams p{};
  p.tokens = tokens;
  p.pages = pages;
  p.heads = heads;
  p.dim = dim;
  p.page = page;
  p.slots = slots;
  p.k = k;
  p.v = v;
  p.k_token = k_token;
  p.k_head = k_head;
  p.v_token = v_token;
  p.v_head = v_head;
  p.k_codes = (uint8_t *)k_codes;
  p.k_scales = (uint8_t *)k_scales;
  p.v_codes = (uint8_t *)v_codes;
  p.v_scales = (uint8_t *)v_scales;
  return status_of(launch_cache_write(p, dtype, bits, (hipStream_t)stream));
}

int kv_cache_read(int64_t tokens, int32_t heads, int32_t dim, int32_t dtype, const int32_t *slots,
                  int64_t pages, int32_t page, int32_t bits, const void *k_codes,
                  const void *k_scales, const void *v_codes, const void *v_scales, void *k,
                  int64_t k_token, int64_t k_head, void *v, int64_t v_token, int64_t v_head,
                  void *stream) {
  if (tokens < 0 || tokens > INT32_MAX || !float_dtype(dtype)) return DLRM_ERR_SHAPE;
  const int bad = cache_shape(heads, dim, pages, page, bits);
  if (bad) return bad;
  if (!out_rows(tokens, heads, dim, k_token, k_head) ||
      !out_rows(tokens, heads, dim, v_token, v_head))
    return DLRM_ERR_SHAPE;
  if (tokens == 0) return DLRM_OK;
  if (!k || !v || !slots || !k_codes || !k_scales || !v_codes || !v_scales) return DLRM_ERR_NULL;
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_scales) || !aligned16(v_scales))
    return DLRM_ERR_UNSUPPORTED;
  CacheParams p{};
  p.tokens = tokens;
  p.pages = pages;
  p.heads = heads;
  p.dim = dim;
  p.page = page;
  p.slots = slots;
  p.out_k = k;
  p.out_v = v;
  p.k_token = k_token;
  p.k_head = k_head;
  p.v_token = v_token;
  p.v_head = v_head;
  p.k_codes = (uint8_t *)const_cast<void *>(k_codes);
  p.k_scales = (uint8_t *)const_cast<void *>(k_scales);
  p.v_codes = (uint8_t *)const_cast<void *>(v_codes);
  p.v_scales = (uint8_t *)const_cast<void *>(v_scales);
  return status_of(launch_cache_read(p, dtype, bits, (hipStream_t)stream));
}

size_t attention_cached_workspace_bytes(int64_t batch, int32_t heads, int32_t kv_heads, int32_t dim,
                                        int64_t max_pages, int32_t page) {
  if (batch < 1 || batch > INT32_MAX || kv_heads < 1 || heads < kv_heads || heads > kMaxHeads ||
      heads % kv_heads || max_pages < 0 || max_pages > INT32_MAX ||
      cache_shape(kv_heads, dim, 1, page, 8))
    return 0;
  return cached_workspace(batch, heads, kv_heads, dim, max_pages, page);
}

int attention_cached(int64_t batch, int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype,
                     const void *q, int64_t q_token, int64_t q_head, int64_t pages, int32_t page,
                     int32_t bits, const void *k_codes, const void *k_scales, const void *v_codes,
                     const void *v_scales, const int32_t *table, int64_t ld_table,
                     int64_t max_pages, const int32_t *lengths, float scale, void *out,
                     int64_t o_token, int64_t o_head, void *workspace, size_t workspace_bytes,
                     void *stream) {
  if (batch < 0 || batch > INT32_MAX || heads < 1 || heads > kMaxHeads || kv_heads < 1 ||
      kv_heads > heads || heads % kv_heads || !float_dtype(dtype) || max_pages < 0 ||
      max_pages > INT32_MAX || ld_table < 0 || !scale_of_scores(scale))
    return DLRM_ERR_SHAPE;
  const int bad = cache_shape(kv_heads, dim, pages, page, bits);
  if (bad) return bad;
  if (!in_rows(q_token, q_head) || !out_rows(batch, heads, dim, o_token, o_head))
    return DLRM_ERR_SHAPE;
  if (batch == 0) return DLRM_OK;
  if (!q || !k_codes || !k_scales || !v_codes || !v_scales || (max_pages > 0 && !table) ||
      !lengths || !out)
    return DLRM_ERR_NULL;
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_scales) || !aligned16(v_scales))
    return DLRM_ERR_UNSUPPORTED;
  const size_t need = cached_workspace(batch, heads, kv_heads, dim, max_pages, page);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return DLRM_ERR_WORKSPACE;
  CachedParams p{};
  p.batch = batch;
  p.pages = pages;
  p.max_pages = max_pages;
  p.heads = heads;
  p.group = heads / kv_heads;
  p.page = page;
  p.q = {q, q_token, q_head};
  p.k_codes = (const uint8_t *)k_codes;
  p.k_scales = (const uint8_t *)k_scales;
  p.v_codes = (const uint8_t *)v_codes;
  p.v_scales = (const uint8_t *)v_scales;
  p.table = table;
  p.ld_table = ld_table;
  p.lengths = lengths;
  p.scale = scale;
  p.out = {out, o_token, o_head};
  return status_of(launch_cached(p, dtype, dim, bits, workspace, (hipStream_t)stream));
}

}  // extern "C"

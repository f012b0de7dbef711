// api_attn.cu -- the C ABI of the paged key-value cache and the attention:
// argument validation, workspace sizing, dispatch to the kernel launchers.
// Every error is found on the host before anything is launched.
#include <cmath>

#include "internal.h"

namespace {

#define QRE_FAIL(code, ...)             \
  do {                                  \
    qre::set_error_message(__VA_ARGS__); \
    return code;                        \
  } while (0)

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

#define QRE_NEED(p)                                                                     \
  do {                                                                                  \
    if (!(p)) QRE_FAIL(QRE_ERR_INVALID_ARG, "%s is NULL", #p);                          \
    if (misaligned(p)) QRE_FAIL(QRE_ERR_MISALIGNED, "%s is not 16-byte aligned", #p);   \
  } while (0)
#define QRE_MAY(p)                                                                              \
  do {                                                                                          \
    if ((p) && misaligned(p)) QRE_FAIL(QRE_ERR_MISALIGNED, "%s is not 16-byte aligned", #p);    \
  } while (0)

constexpr int kMaxCount = 1 << 24;

bool head_dim_ok(int d) { return d == 64 || d == 128; }

bool quantized(int dtype) { return dtype == QRE_E4M3 || dtype == QRE_E2M1; }

qre_status check_cache(const qre_kv_cache* c, bool scales) {
  if (!c) QRE_FAIL(QRE_ERR_INVALID_ARG, "cache is NULL");
  if (c->n_layers <= 0 || c->n_pages <= 0 || c->n_kv_heads <= 0 || c->page_size <= 0 || c->head_dim <= 0 ||
      c->max_seqs <= 0 || c->max_pages <= 0)
    QRE_FAIL(QRE_ERR_INVALID_ARG,
             "cache sizes must be positive (layers %d, pages %d, KV heads %d, page size %d, head dim %d, seqs %d, "
             "pages per seq %d)",
             c->n_layers, c->n_pages, c->n_kv_heads, c->page_size, c->head_dim, c->max_seqs, c->max_pages);
  if (c->dtype != QRE_BF16 && c->dtype != QRE_FP16 && !quantized(c->dtype))
    QRE_FAIL(QRE_ERR_INVALID_ARG, "cache dtype %d is not a qre_dtype", c->dtype);
  if (!head_dim_ok(c->head_dim)) QRE_FAIL(QRE_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", c->head_dim);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "page_size %d is not a power of two from 16 to 256", c->page_size);
  if (c->n_kv_heads > qre::kKvMaxHeads) QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_kv_heads %d > %d", c->n_kv_heads, qre::kKvMaxHeads);
  if (c->n_pages >= kMaxCount || c->max_seqs >= kMaxCount || c->max_pages >= kMaxCount || c->n_layers >= kMaxCount)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "cache sizes must be below 2^24");
  if ((long long)c->max_pages * c->page_size > 0x7fffffffll)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "max_pages * page_size = %lld positions do not fit 31 bits",
             (long long)c->max_pages * c->page_size);
  QRE_NEED(c->k);
  QRE_NEED(c->v);
  QRE_NEED(c->page_table);
  QRE_NEED(c->seq_len);
  QRE_NEED(c->ref_count);
  if (scales) {
    if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u)
      QRE_FAIL(QRE_ERR_MISALIGNED, "k_scale or v_scale is not 4-byte aligned");
    if (!quantized(c->dtype) && (c->k_scale || c->v_scale))
      QRE_FAIL(QRE_ERR_INVALID_ARG, "k_scale and v_scale belong to a QRE_E4M3 or QRE_E2M1 cache");
  }
  return QRE_OK;
}

qre_status check_count(int32_t n, const char* name) {
  if (n < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "%s = %d is negative", name, n);
  if (n > qre::kKvMaxRequests) QRE_FAIL(QRE_ERR_UNSUPPORTED, "%s = %d > %d", name, n, qre::kKvMaxRequests);
  return QRE_OK;
}

qre_status check_layer(const qre_kv_cache* c, int32_t layer) {
  if (layer < 0 || layer >= c->n_layers)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "layer %d not in [0, %d)", layer, c->n_layers);
  return QRE_OK;
}

qre_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) QRE_FAIL(QRE_ERR_INVALID_ARG, "workspace is NULL");
  if (misaligned(ws)) QRE_FAIL(QRE_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  if (have < need) QRE_FAIL(QRE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return QRE_OK;
}

qre_status check_stride(int64_t s, const char* name) {
  if (s < 0 || s % 8) QRE_FAIL(QRE_ERR_INVALID_ARG, "%s = %lld is not a non-negative multiple of 8 elements", name,
                               (long long)s);
  if (s >= (1ll << 38)) QRE_FAIL(QRE_ERR_UNSUPPORTED, "%s = %lld elements is too large", name, (long long)s);
  return QRE_OK;
}

#define QRE_STRIDE(owner, f)                          \
  do {                                                    \
    const qre_status e_ = check_stride((owner)->f, #f);   \
    if (e_ != QRE_OK) return e_;                          \
  } while (0)

qre_status check_rows(const qre_kv_rows* rows, const qre_kv_cache* cache) {
  if (!rows) QRE_FAIL(QRE_ERR_INVALID_ARG, "rows is NULL");
  if (rows->dtype != QRE_BF16 && rows->dtype != QRE_FP16)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "rows dtype %d is not QRE_BF16 or QRE_FP16", rows->dtype);
  if (!quantized(cache->dtype) && cache->dtype != rows->dtype)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "rows of dtype %d into a cache of dtype %d", rows->dtype, cache->dtype);
  if (rows->reserved != 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "rows reserved field is %d, must be 0", rows->reserved);
  QRE_STRIDE(rows, k_token);
  QRE_STRIDE(rows, k_head);
  QRE_STRIDE(rows, v_token);
  QRE_STRIDE(rows, v_head);
  return QRE_OK;
}

qre_status check_rope(const qre_rope* r, bool cache) {
  if (!r) QRE_FAIL(QRE_ERR_INVALID_ARG, "rope is NULL");
  if (r->n_heads <= 0 || r->n_kv_heads <= 0 || r->head_dim <= 0)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "rope sizes must be positive (heads %d, KV heads %d, head dim %d)", r->n_heads,
             r->n_kv_heads, r->head_dim);
  if (r->dtype != QRE_BF16 && r->dtype != QRE_FP16)
    QRE_FAIL(quantized(r->dtype) ? QRE_ERR_UNSUPPORTED : QRE_ERR_INVALID_ARG, "rope dtype %d is not QRE_BF16 or QRE_FP16",
             r->dtype);
  if (!head_dim_ok(r->head_dim)) QRE_FAIL(QRE_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", r->head_dim);
  if (r->n_heads > 1024 || r->n_kv_heads > qre::kKvMaxHeads)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_heads %d > 1024 or n_kv_heads %d > %d", r->n_heads, r->n_kv_heads, qre::kKvMaxHeads);
  if (r->rot_dim < 0 || r->rot_dim > r->head_dim)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "rot_dim %d not in [0, %d]", r->rot_dim, r->head_dim);
  if (r->rot_dim % 16) QRE_FAIL(QRE_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16", r->rot_dim);
  if (!(std::isfinite(r->eps) && r->eps >= 0.0f)) QRE_FAIL(QRE_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (r->reserved != 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "rope reserved field is %d, must be 0", r->reserved);
  if (r->rot_dim > 0) QRE_NEED(r->inv_freq);
  QRE_MAY(r->q_norm);
  QRE_MAY(r->k_norm);
  QRE_STRIDE(r, q_token);
  QRE_STRIDE(r, q_head);
  QRE_STRIDE(r, k_token);
  QRE_STRIDE(r, k_head);
  QRE_STRIDE(r, qo_token);
  QRE_STRIDE(r, qo_head);
  QRE_STRIDE(r, ko_token);
  QRE_STRIDE(r, ko_head);
  if (cache) {
    QRE_STRIDE(r, v_token);
    QRE_STRIDE(r, v_head);
  }
  return QRE_OK;
}

// Rows of an output that lie on one another would be written in any order.
qre_status check_apart(int64_t token, int64_t head, int32_t tokens, int32_t heads, const char* name) {
  if ((tokens > 1 && token == 0) || (heads > 1 && head == 0))
    QRE_FAIL(QRE_ERR_INVALID_ARG, "rows of %s lie on one another (strides %lld and %lld)", name, (long long)token,
             (long long)head);
  return QRE_OK;
}

qre_status check_attn(const qre_attn* a) {
  if (!a) QRE_FAIL(QRE_ERR_INVALID_ARG, "attn is NULL");
  if (a->n_heads <= 0 || a->n_kv_heads <= 0 || a->head_dim <= 0)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "attention sizes must be positive (heads %d, KV heads %d, head dim %d)", a->n_heads,
             a->n_kv_heads, a->head_dim);
  if (a->n_heads % a->n_kv_heads)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "n_heads %d is not a multiple of n_kv_heads %d", a->n_heads, a->n_kv_heads);
  if (a->dtype != QRE_BF16 && a->dtype != QRE_FP16)
    QRE_FAIL(quantized(a->dtype) ? QRE_ERR_UNSUPPORTED : QRE_ERR_INVALID_ARG,
             "attention dtype %d is not QRE_BF16 or QRE_FP16", a->dtype);
  if (!head_dim_ok(a->head_dim)) QRE_FAIL(QRE_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", a->head_dim);
  if (a->n_heads > 1024 || a->n_kv_heads > 256)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_heads %d > 1024 or n_kv_heads %d > 256", a->n_heads, a->n_kv_heads);
  if (!(std::isfinite(a->scale) && a->scale > 0.0f))
    QRE_FAIL(QRE_ERR_INVALID_ARG, "scale must be finite and positive");
  if (a->window < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "window %d is negative", a->window);
  if (a->window > 0 && !a->causal) QRE_FAIL(QRE_ERR_INVALID_ARG, "a window needs causal attention");
  if (a->reserved != 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "attn reserved field is %d, must be 0", a->reserved);
  QRE_STRIDE(a, q_token);
  QRE_STRIDE(a, q_head);
  QRE_STRIDE(a, o_token);
  QRE_STRIDE(a, o_head);
  return QRE_OK;
}

qre_status check_pair(const qre_attn* a, const qre_kv_cache* c) {
  if (a->n_kv_heads != c->n_kv_heads || a->head_dim != c->head_dim)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "attention (%d KV heads of %d) and cache (%d of %d) differ", a->n_kv_heads,
             a->head_dim, c->n_kv_heads, c->head_dim);
  if (!quantized(c->dtype) && c->dtype != a->dtype)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "attention dtype %d with a cache of dtype %d", a->dtype, c->dtype);
  return QRE_OK;
}

qre_status done(cudaError_t e, const char* what) {
  if (e != cudaSuccess) QRE_FAIL(QRE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  qre::set_error_message("%s", "");
  return QRE_OK;
}

cudaStream_t cu_stream(qre_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

#define QRE_TRY(expr)                       \
  do {                                      \
    const qre_status e_ = (expr);           \
    if (e_ != QRE_OK) return e_;            \
  } while (0)

extern "C" {

qre_status qre_kv_workspace_size(const qre_kv_cache* cache, size_t* bytes) {
  QRE_TRY(check_cache(cache, false));
  if (!bytes) QRE_FAIL(QRE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = qre::kv_ws_bytes(*cache);
  return done(cudaSuccess, "");
}

qre_status qre_kv_reserve(const qre_kv_cache* cache, int32_t n, const int32_t* seqs, const int32_t* n_new,
                          void* workspace, size_t workspace_bytes, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_count(n, "n"));
  if (n == 0) return QRE_OK;
  QRE_NEED(seqs);
  QRE_NEED(n_new);
  QRE_TRY(check_ws(workspace, workspace_bytes, qre::kv_ws_bytes(*cache)));
  return done(qre::launch_kv_reserve(*cache, n, seqs, n_new, workspace, qre::device_status_word(), cu_stream(stream)),
              "qre_kv_reserve launch");
}

qre_status qre_kv_write(const qre_kv_cache* cache, int32_t layer, const qre_kv_rows* rows, int32_t n_tokens,
                        const int32_t* token_seq, const int32_t* token_pos, const void* k, const void* v,
                        qre_stream_t stream) {
  QRE_TRY(check_cache(cache, true));
  QRE_TRY(check_layer(cache, layer));
  QRE_TRY(check_rows(rows, cache));
  if (n_tokens < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "n_tokens = %d is negative", n_tokens);
  if (n_tokens >= kMaxCount) QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_tokens = %d is not below 2^24", n_tokens);
  if (n_tokens == 0) return QRE_OK;
  QRE_NEED(token_seq);
  QRE_NEED(token_pos);
  QRE_NEED(k);
  QRE_NEED(v);
  return done(qre::launch_kv_write(*cache, layer, *rows, n_tokens, token_seq, token_pos, k, v,
                                   qre::device_status_word(), cu_stream(stream)),
              "qre_kv_write launch");
}

qre_status qre_kv_read(const qre_kv_cache* cache, int32_t layer, const qre_kv_rows* rows, int32_t n,
                       const int32_t* seqs, const int32_t* first, const int32_t* cu, int32_t total, void* k, void* v,
                       qre_stream_t stream) {
  QRE_TRY(check_cache(cache, true));
  QRE_TRY(check_layer(cache, layer));
  QRE_TRY(check_rows(rows, cache));
  QRE_TRY(check_count(n, "n"));
  if (total < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "total = %d is negative", total);
  if (total >= kMaxCount) QRE_FAIL(QRE_ERR_UNSUPPORTED, "total = %d is not below 2^24", total);
  QRE_TRY(check_apart(rows->k_token, rows->k_head, total, cache->n_kv_heads, "k"));
  QRE_TRY(check_apart(rows->v_token, rows->v_head, total, cache->n_kv_heads, "v"));
  if (n == 0 || total == 0) return QRE_OK;
  if (!seqs && n > cache->max_seqs)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "n = %d without seqs, and the cache has %d sequences", n, cache->max_seqs);
  QRE_MAY(seqs);
  QRE_MAY(first);
  QRE_NEED(cu);
  QRE_NEED(k);
  QRE_NEED(v);
  return done(qre::launch_kv_read(*cache, layer, *rows, n, seqs, first, cu, total, k, v, qre::device_status_word(), cu_stream(stream)),
              "qre_kv_read launch");
}

qre_status qre_qk_norm_rope(const qre_rope* rope, int32_t n_tokens, const int32_t* token_pos, const void* q,
                            const void* k, void* q_out, void* k_out, qre_stream_t stream) {
  QRE_TRY(check_rope(rope, false));
  if (n_tokens < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "n_tokens = %d is negative", n_tokens);
  if (n_tokens >= kMaxCount) QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_tokens = %d is not below 2^24", n_tokens);
  QRE_TRY(check_apart(rope->qo_token, rope->qo_head, n_tokens, rope->n_heads, "q_out"));
  QRE_TRY(check_apart(rope->ko_token, rope->ko_head, n_tokens, rope->n_kv_heads, "k_out"));
  if (n_tokens == 0) return QRE_OK;
  QRE_NEED(token_pos);
  QRE_NEED(q);
  QRE_NEED(k);
  QRE_NEED(q_out);
  QRE_NEED(k_out);
  return done(qre::launch_qk_rope(*rope, nullptr, 0, n_tokens, nullptr, token_pos, q, k, nullptr, q_out, k_out,
                                  qre::device_status_word(), cu_stream(stream)),
              "qre_qk_norm_rope launch");
}

qre_status qre_kv_write_rope(const qre_kv_cache* cache, int32_t layer, const qre_rope* rope, int32_t n_tokens,
                             const int32_t* token_seq, const int32_t* token_pos, const void* q, const void* k,
                             const void* v, void* q_out, void* k_out, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, true));
  QRE_TRY(check_layer(cache, layer));
  QRE_TRY(check_rope(rope, true));
  if (rope->n_kv_heads != cache->n_kv_heads || rope->head_dim != cache->head_dim)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "rope (%d KV heads of %d) and cache (%d of %d) differ", rope->n_kv_heads, rope->head_dim,
             cache->n_kv_heads, cache->head_dim);
  if (!quantized(cache->dtype) && cache->dtype != rope->dtype)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "rows of dtype %d into a cache of dtype %d", rope->dtype, cache->dtype);
  if (n_tokens < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "n_tokens = %d is negative", n_tokens);
  if (n_tokens >= kMaxCount) QRE_FAIL(QRE_ERR_UNSUPPORTED, "n_tokens = %d is not below 2^24", n_tokens);
  QRE_TRY(check_apart(rope->qo_token, rope->qo_head, n_tokens, rope->n_heads, "q_out"));
  if (k_out) QRE_TRY(check_apart(rope->ko_token, rope->ko_head, n_tokens, rope->n_kv_heads, "k_out"));
  if (n_tokens == 0) return QRE_OK;
  QRE_NEED(token_seq);
  QRE_NEED(token_pos);
  QRE_NEED(q);
  QRE_NEED(k);
  QRE_NEED(v);
  QRE_NEED(q_out);
  QRE_MAY(k_out);
  return done(qre::launch_qk_rope(*rope, cache, layer, n_tokens, token_seq, token_pos, q, k, v, q_out, k_out,
                                  qre::device_status_word(), cu_stream(stream)),
              "qre_kv_write_rope launch");
}

qre_status qre_kv_fork(const qre_kv_cache* cache, int32_t n, const int32_t* src, const int32_t* dst, void* workspace,
                       size_t workspace_bytes, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_count(n, "n"));
  if (n == 0) return QRE_OK;
  QRE_NEED(src);
  QRE_NEED(dst);
  QRE_TRY(check_ws(workspace, workspace_bytes, qre::kv_ws_bytes(*cache)));
  return done(qre::launch_kv_fork(*cache, n, src, dst, workspace, qre::device_status_word(), cu_stream(stream)),
              "qre_kv_fork launch");
}

qre_status qre_kv_free(const qre_kv_cache* cache, int32_t n, const int32_t* seqs, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_count(n, "n"));
  if (n == 0) return QRE_OK;
  QRE_NEED(seqs);
  return done(qre::launch_kv_free(*cache, n, seqs, qre::device_status_word(), cu_stream(stream)), "qre_kv_free launch");
}

qre_status qre_kv_compact(const qre_kv_cache* cache, int32_t* page_table_out, int32_t* ref_count_out, int32_t* n_live,
                          void* workspace, size_t workspace_bytes, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, false));
  QRE_NEED(page_table_out);
  QRE_NEED(ref_count_out);
  QRE_NEED(n_live);
  QRE_TRY(check_ws(workspace, workspace_bytes, qre::kv_ws_bytes(*cache)));
  return done(qre::launch_kv_compact(*cache, page_table_out, ref_count_out, n_live, workspace,
                                     qre::device_status_word(), cu_stream(stream)),
              "qre_kv_compact launch");
}

qre_status qre_attn_prefill(const qre_attn* attn, int32_t n_seqs, int32_t total_q, int32_t total_k,
                            const int32_t* cu_q, const int32_t* cu_k, const void* q, const void* k, const void* v,
                            void* o, float* lse, qre_stream_t stream) {
  QRE_TRY(check_attn(attn));
  QRE_STRIDE(attn, k_token);
  QRE_STRIDE(attn, k_head);
  QRE_STRIDE(attn, v_token);
  QRE_STRIDE(attn, v_head);
  QRE_TRY(check_count(n_seqs, "n_seqs"));
  if (total_q < 0 || total_k < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "total_q %d or total_k %d is negative", total_q, total_k);
  if (total_q >= kMaxCount || total_k >= kMaxCount)
    QRE_FAIL(QRE_ERR_UNSUPPORTED, "total_q %d and total_k %d must be below 2^24", total_q, total_k);
  if (n_seqs == 0 || total_q == 0) return QRE_OK;
  QRE_NEED(cu_q);
  QRE_NEED(cu_k);
  QRE_NEED(q);
  if (total_k > 0) {
    QRE_NEED(k);
    QRE_NEED(v);
  }
  QRE_NEED(o);
  QRE_MAY(lse);
  return done(qre::launch_attn_prefill(*attn, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse,
                                       qre::device_status_word(), cu_stream(stream)),
              "qre_attn_prefill launch");
}

qre_status qre_attn_decode_workspace_size(const qre_attn* attn, const qre_kv_cache* cache, int32_t n, size_t* bytes) {
  QRE_TRY(check_attn(attn));
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_pair(attn, cache));
  QRE_TRY(check_count(n, "n"));
  if (!bytes) QRE_FAIL(QRE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = qre::attn_decode_ws_bytes(*attn, *cache, n);
  return done(cudaSuccess, "");
}

qre_status qre_attn_decode(const qre_attn* attn, const qre_kv_cache* cache, int32_t layer, int32_t n,
                           const int32_t* seqs, int32_t max_len, const void* q, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, qre_stream_t stream) {
  QRE_TRY(check_attn(attn));
  QRE_TRY(check_cache(cache, true));
  QRE_TRY(check_pair(attn, cache));
  QRE_TRY(check_layer(cache, layer));
  QRE_TRY(check_count(n, "n"));
  if (!attn->causal) QRE_FAIL(QRE_ERR_INVALID_ARG, "qre_attn_decode is causal: attn->causal is 0");
  if (max_len < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "max_len = %d is negative", max_len);
  if (n == 0) return QRE_OK;
  if (!seqs && n > cache->max_seqs)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "n = %d without seqs, and the cache has %d sequences", n, cache->max_seqs);
  QRE_MAY(seqs);
  QRE_NEED(q);
  QRE_NEED(o);
  QRE_MAY(lse);
  QRE_TRY(check_ws(workspace, workspace_bytes, qre::attn_decode_ws_bytes(*attn, *cache, n)));
  return done(qre::launch_attn_decode(*attn, *cache, layer, n, seqs, max_len, q, o, lse, workspace,
                                      qre::device_status_word(), cu_stream(stream)),
              "qre_attn_decode launch");
}

qre_status qre_kv_common_len(const qre_kv_cache* cache, int32_t n, const int32_t* seqs, int32_t n_groups,
                             const int32_t* cu_group, int32_t* common_len, qre_stream_t stream) {
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_count(n, "n"));
  QRE_TRY(check_count(n_groups, "n_groups"));
  if (n_groups == 0) return QRE_OK;
  if (!seqs && n > cache->max_seqs)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "n = %d without seqs, and the cache has %d sequences", n, cache->max_seqs);
  QRE_MAY(seqs);
  QRE_NEED(cu_group);
  QRE_NEED(common_len);
  return done(qre::launch_kv_common_len(*cache, n, seqs, n_groups, cu_group, common_len, qre::device_status_word(),
                                        cu_stream(stream)),
              "qre_kv_common_len launch");
}

qre_status qre_attn_decode_shared_workspace_size(const qre_attn* attn, const qre_kv_cache* cache, int32_t n,
                                                 int32_t n_groups, size_t* bytes) {
  QRE_TRY(check_attn(attn));
  QRE_TRY(check_cache(cache, false));
  QRE_TRY(check_pair(attn, cache));
  QRE_TRY(check_count(n, "n"));
  QRE_TRY(check_count(n_groups, "n_groups"));
  if (!bytes) QRE_FAIL(QRE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = qre::attn_shared_ws_bytes(*attn, *cache, n, n_groups);
  return done(cudaSuccess, "");
}

qre_status qre_attn_decode_shared(const qre_attn* attn, const qre_kv_cache* cache, int32_t layer, int32_t n,
                                  const int32_t* seqs, int32_t n_groups, const int32_t* cu_group,
                                  const int32_t* common_len, int32_t max_len, const void* q, void* o, float* lse,
                                  void* workspace, size_t workspace_bytes, qre_stream_t stream) {
  QRE_TRY(check_attn(attn));
  QRE_TRY(check_cache(cache, true));
  QRE_TRY(check_pair(attn, cache));
  QRE_TRY(check_layer(cache, layer));
  QRE_TRY(check_count(n, "n"));
  QRE_TRY(check_count(n_groups, "n_groups"));
  if (!attn->causal) QRE_FAIL(QRE_ERR_INVALID_ARG, "qre_attn_decode_shared is causal: attn->causal is 0");
  if (max_len < 0) QRE_FAIL(QRE_ERR_INVALID_ARG, "max_len = %d is negative", max_len);
  if (n == 0) return QRE_OK;
  if (!seqs && n > cache->max_seqs)
    QRE_FAIL(QRE_ERR_INVALID_ARG, "n = %d without seqs, and the cache has %d sequences", n, cache->max_seqs);
  QRE_MAY(seqs);
  if (n_groups > 0) {
    QRE_NEED(cu_group);
    QRE_NEED(common_len);
  }
  QRE_NEED(q);
  QRE_NEED(o);
  QRE_MAY(lse);
  QRE_TRY(check_ws(workspace, workspace_bytes, qre::attn_shared_ws_bytes(*attn, *cache, n, n_groups)));
  return done(qre::launch_attn_decode_shared(*attn, *cache, layer, n, seqs, n_groups, cu_group, common_len, max_len, q, o,
                                             lse, workspace, qre::device_status_word(), cu_stream(stream)),
              "qre_attn_decode_shared launch");
}

}  // extern "C"

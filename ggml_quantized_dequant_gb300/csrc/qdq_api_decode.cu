// C-ABI boundary of the decode-step operators (norm, 8-bit cache, attention, log
// probabilities): argument checks and status codes, as in qdq_api.cu.
#include <cmath>

#include "qdq_types.cuh"

using namespace qdq;

namespace {

// A NULL pointer is refused only where the call has something to do: an empty tensor's is NULL.

// A byte range, or rows of `row` bytes `stride` bytes apart (stride 0: one range).
struct Span {
  const void *p;
  size_t n;
  size_t stride = 0, row = 0;
};
Span span(const void *p, int64_t rows, int64_t stride, int64_t row, int eb) {
  if (!p || rows <= 0) return {p, 0};
  return {p, size_t((rows - 1) * stride + row) * eb, rows > 1 ? size_t(stride) * eb : 0, size_t(row) * eb};
}
// Rows of one stride (or one row among another's) that lie beside one another, as slices of one wide
// buffer do, do not clash; rows of different strides whose spans overlap count as if they did.
bool clash(const Span &a, const Span &b) {
  if (!a.p || !b.p || !overlaps(a.p, a.n, b.p, b.n)) return false;
  const size_t s = a.stride ? a.stride : b.stride;
  if (s == 0 || (a.stride && b.stride && a.stride != b.stride)) return true;
  const size_t la = a.stride ? a.row : a.n, lb = b.stride ? b.row : b.n;
  const intptr_t off = (reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) % intptr_t(s);
  const size_t d = size_t(off < 0 ? off + intptr_t(s) : off);  // how far b's rows start behind a's
  return d < la || d + lb > s;
}

bool dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

int check_pool(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *table,
               int table_stride, int n_seqs, bool nothing) {
  if (!nothing && (!pages || !table)) return QDQ_ERR_NULL;
  if (n_pages < 1 || page_tokens < QDQ_KV_BLOCK || page_tokens % QDQ_KV_BLOCK || n_kv < 1 || head_dim < 1 ||
      table_stride < 1 || n_seqs < 0)
    return QDQ_ERR_DIMS;
  if (!dim_ok(head_dim) || page_tokens > 65536 || n_kv > 65536) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(pages, 128) || !aligned(table, 4)) return QDQ_ERR_ALIGN;
  return QDQ_OK;
}

size_t page_bytes(int page_tokens, int n_kv, int head_dim) { return size_t(n_kv) * size_t(kv_record_bytes(page_tokens, head_dim)); }

int check_rows(const void *p, int64_t stride, int64_t row, int type) {
  if (stride < row) return QDQ_ERR_DIMS;
  if (!aligned(p, 16) || (stride * type_bytes(type)) % 16) return QDQ_ERR_ALIGN;
  return QDQ_OK;
}

// qdq_kv_attention, and with parent qdq_kv_tree_attention.
int attention(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table, int table_stride,
              const int *kv_len, const int *cu_q, const int *parent, int n_seqs, int max_q, int max_kv_len, int n_heads, const void *q,
              int64_t q_stride, void *out, int64_t out_stride, float *lse, const float *slopes, float scale, float softcap,
              int window, int type, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  const bool nothing = n_seqs == 0 || max_q == 0;
  if (!nothing && (!kv_len || !q || !out || !workspace)) return QDQ_ERR_NULL;
  int rc = check_pool(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, n_seqs, nothing);
  if (rc != QDQ_OK) return rc;
  if (!type_ok(type) || max_q < 0 || (!cu_q && max_q != 1) || max_kv_len < 0 || n_heads < 1 || n_heads % n_kv || window < 0 ||
      !std::isfinite(scale) || !(softcap >= 0.f) || !std::isfinite(softcap))
    return QDQ_ERR_DIMS;
  if (max_kv_len > QDQ_MAX_KV_LEN || max_q > (1 << 20) || n_heads / n_kv > 1024) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(kv_len, 4) || !aligned(cu_q, 4) || !aligned(parent, 4) || !aligned(lse, 4) || !aligned(slopes, 4) || !aligned(workspace, 256))
    return QDQ_ERR_ALIGN;
  const int64_t width = int64_t(n_heads) * head_dim;
  if ((rc = check_rows(q, q_stride, width, type)) != QDQ_OK || (rc = check_rows(out, out_stride, width, type)) != QDQ_OK) return rc;
  if (nothing) return QDQ_OK;
  const int64_t known = cu_q ? 1 : n_seqs;  // query rows the host can count on
  const int eb = type_bytes(type);
  const Span so = span(out, known, out_stride, width, eb), sl = span(lse, known, n_heads, n_heads, 4);
  const Span sws{workspace, workspace_bytes}, sq = span(q, known, q_stride, width, eb);
  const Span in[7] = {{pages, size_t(n_pages) * page_bytes(page_tokens, n_kv, head_dim)},
                      {page_table, size_t(n_seqs) * table_stride * 4},
                      {kv_len, size_t(n_seqs) * 4},
                      {cu_q, size_t(n_seqs + 1) * 4},
                      {slopes, size_t(n_heads) * 4},
                      sq,
                      {parent, size_t(known) * 4}};
  for (const Span &i : in)
    if (clash(i, so) || clash(i, sl) || clash(i, sws)) return QDQ_ERR_ALIAS;
  if (clash(so, sl) || clash(so, sws) || clash(sl, sws)) return QDQ_ERR_ALIAS;
  const size_t need = kv_attention_workspace_bytes(n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim, parent != nullptr);
  if (workspace_bytes < need) return QDQ_ERR_SCRATCH;
  const KvPool c{static_cast<uint8_t *>(const_cast<void *>(pages)), page_table, n_pages, page_tokens, n_kv, table_stride};
  return launch_kv_attention(c, head_dim, kv_len, cu_q, parent, n_seqs, max_q, max_kv_len, n_heads, q, q_stride, out, out_stride, lse,
                             slopes, scale, softcap, window, type, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

int qdq_rms_norm(const void *x, const void *residual, const float *weight, void *sum_out, void *out, void *q8_out,
                 int type, int rows, int n, long long x_stride, long long residual_stride, long long sum_stride,
                 long long out_stride, float eps, cudaStream_t stream) {
  if (rows != 0 && (!x || (!out && !q8_out))) return QDQ_ERR_NULL;
  if (!type_ok(type) || rows < 0 || n < 1 || !(eps >= 0.f) || (q8_out && n % 32)) return QDQ_ERR_DIMS;
  if (x_stride < n || (residual && residual_stride < n) || (sum_out && sum_stride < n) || (out && out_stride < n))
    return QDQ_ERR_DIMS;
  if (n > QDQ_MAX_NORM_N) return QDQ_ERR_UNSUPPORTED;
  const int eb = type_bytes(type);
  if (!aligned(x, eb) || !aligned(residual, eb) || !aligned(weight, 4) || !aligned(sum_out, eb) || !aligned(out, eb) ||
      !aligned(q8_out, 16))
    return QDQ_ERR_ALIGN;
  if (rows == 0) return QDQ_OK;
  const Span sx = span(x, rows, x_stride, n, eb), sr = span(residual, rows, residual_stride, n, eb);
  const Span sw = span(weight, 1, n, n, 4), ss = span(sum_out, rows, sum_stride, n, eb);
  const Span so = span(out, rows, out_stride, n, eb), sq = span(q8_out, 1, 0, q8_out ? int64_t(rows) * (n / 32) * 34 : 0, 1);
  // in place: exactly the same rows as x or the residual
  auto same = [](const Span &o, int64_t os, const Span &i, int64_t is) { return o.p == i.p && os == is; };
  if ((clash(ss, sx) && !same(ss, sum_stride, sx, x_stride)) || (clash(ss, sr) && !same(ss, sum_stride, sr, residual_stride)) ||
      (clash(so, sx) && !same(so, out_stride, sx, x_stride)) || (clash(so, sr) && !same(so, out_stride, sr, residual_stride)))
    return QDQ_ERR_ALIAS;
  if (clash(ss, sw) || clash(so, sw) || clash(ss, so) || clash(sq, sx) || clash(sq, sr) || clash(sq, sw) || clash(sq, ss) ||
      clash(sq, so))
    return QDQ_ERR_ALIAS;
  return launch_rms_norm(x, residual, weight, sum_out, out, q8_out, type, rows, n, x_stride, residual_stride, sum_stride,
                         out_stride, eps, stream);
}

size_t qdq_kv_page_bytes(int page_tokens, int n_kv, int head_dim) {
  if (page_tokens < QDQ_KV_BLOCK || page_tokens % QDQ_KV_BLOCK || page_tokens > 65536 || n_kv < 1 || n_kv > 65536 ||
      !dim_ok(head_dim))
    return 0;
  return page_bytes(page_tokens, n_kv, head_dim);
}

int qdq_kv_append(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                  int table_stride, const int *kv_len, const int *cu_new, int n_seqs, int max_new, const void *k,
                  const void *v, long long k_stride, long long v_stride, int type, cudaStream_t stream) {
  const bool nothing = n_seqs == 0 || max_new == 0;
  if (!nothing && (!kv_len || !k || !v)) return QDQ_ERR_NULL;
  int rc = check_pool(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, n_seqs, nothing);
  if (rc != QDQ_OK) return rc;
  if (!type_ok(type) || max_new < 0 || (!cu_new && max_new != 1)) return QDQ_ERR_DIMS;
  if (!aligned(kv_len, 4) || !aligned(cu_new, 4)) return QDQ_ERR_ALIGN;
  const int64_t width = int64_t(n_kv) * head_dim;
  if ((rc = check_rows(k, k_stride, width, type)) != QDQ_OK || (rc = check_rows(v, v_stride, width, type)) != QDQ_OK) return rc;
  if (nothing) return QDQ_OK;
  const Span sp{pages, size_t(n_pages) * page_bytes(page_tokens, n_kv, head_dim)};
  const int eb = type_bytes(type);  // at least one row of k and v per call is known to the host
  if (clash(sp, span(k, cu_new ? 1 : n_seqs, k_stride, width, eb)) || clash(sp, span(v, cu_new ? 1 : n_seqs, v_stride, width, eb)) ||
      clash(sp, {page_table, size_t(n_seqs) * table_stride * 4}) || clash(sp, {kv_len, size_t(n_seqs) * 4}) ||
      clash(sp, {cu_new, size_t(n_seqs + 1) * 4}))
    return QDQ_ERR_ALIAS;
  const KvPool c{static_cast<uint8_t *>(pages), page_table, n_pages, page_tokens, n_kv, table_stride};
  return launch_kv_append(c, head_dim, kv_len, cu_new, n_seqs, max_new, k, v, k_stride, v_stride, type, stream);
}

int qdq_kv_read(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                int table_stride, const int *start, const int *cu, int n_seqs, int max_tokens, void *k, void *v,
                long long k_stride, long long v_stride, int type, cudaStream_t stream) {
  const bool nothing = n_seqs == 0 || max_tokens == 0;
  if (!nothing && (!cu || !k || !v)) return QDQ_ERR_NULL;
  int rc = check_pool(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, n_seqs, nothing);
  if (rc != QDQ_OK) return rc;
  if (!type_ok(type) || max_tokens < 0) return QDQ_ERR_DIMS;
  if (!aligned(start, 4) || !aligned(cu, 4)) return QDQ_ERR_ALIGN;
  const int64_t width = int64_t(n_kv) * head_dim;
  if ((rc = check_rows(k, k_stride, width, type)) != QDQ_OK || (rc = check_rows(v, v_stride, width, type)) != QDQ_OK) return rc;
  if (nothing) return QDQ_OK;
  const Span sp{pages, size_t(n_pages) * page_bytes(page_tokens, n_kv, head_dim)};
  const int eb = type_bytes(type);
  const Span sk = span(k, 1, k_stride, width, eb), sv = span(v, 1, v_stride, width, eb);
  const Span in[4] = {sp, {page_table, size_t(n_seqs) * table_stride * 4}, {start, size_t(n_seqs) * 4}, {cu, size_t(n_seqs + 1) * 4}};
  for (const Span &i : in)
    if (clash(i, sk) || clash(i, sv)) return QDQ_ERR_ALIAS;
  if (clash(sk, sv)) return QDQ_ERR_ALIAS;
  const KvPool c{static_cast<uint8_t *>(const_cast<void *>(pages)), page_table, n_pages, page_tokens, n_kv, table_stride};
  return launch_kv_read(c, head_dim, start, cu, n_seqs, max_tokens, k, v, k_stride, v_stride, type, stream);
}

size_t qdq_kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim) {
  if (n_seqs < 1 || max_q < 1 || max_kv_len < 0 || max_kv_len > QDQ_MAX_KV_LEN || n_kv < 1 || n_heads < 1 || n_heads % n_kv || !dim_ok(head_dim) ||
      max_q > (1 << 20) || n_heads / n_kv > 1024)
    return 0;
  const size_t b = kv_attention_workspace_bytes(n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim, false);
  const size_t tree = max_q <= QDQ_MAX_TREE ? kv_attention_workspace_bytes(n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim, true) : 0;
  return b > tree ? b : tree;
}

int qdq_kv_attention(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                     int table_stride, const int *kv_len, const int *cu_q, int n_seqs, int max_q, int max_kv_len,
                     int n_heads, const void *q, long long q_stride, void *out, long long out_stride, float *lse,
                     const float *slopes, float scale, float softcap, int window, int type, void *workspace,
                     size_t workspace_bytes, cudaStream_t stream) {
  return attention(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, kv_len, cu_q, nullptr, n_seqs, max_q,
                   max_kv_len, n_heads, q, q_stride, out, out_stride, lse, slopes, scale, softcap, window, type, workspace,
                   workspace_bytes, stream);
}

size_t qdq_token_logprobs_workspace_bytes(int rows, int n, int k) {
  if (rows < 1 || n < 1 || n > (1 << 30) || k < 0 || k > n || k > QDQ_MAX_TOPK) return 0;
  return token_logprobs_workspace_bytes(rows, n, k);
}

int qdq_token_logprobs(const void *logits, long long row_stride, int type, const int *tokens, int rows, int n, int k,
                       float *logprob, float *entropy, int *top_index, float *top_logprob, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  if (rows != 0 && (!logits || !workspace || !tokens != !logprob || (k > 0 && (!top_index || !top_logprob)))) return QDQ_ERR_NULL;
  if (!type_ok(type) || rows < 0 || n < 1 || k < 0 || k > n || row_stride < n) return QDQ_ERR_DIMS;
  if (k > QDQ_MAX_TOPK || n > (1 << 30)) return QDQ_ERR_UNSUPPORTED;
  const int eb = type_bytes(type);
  if (!aligned(logits, eb) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      (k > 0 && (!aligned(top_index, 4) || !aligned(top_logprob, 4))) || !aligned(workspace, 256))
    return QDQ_ERR_ALIGN;
  if (rows == 0) return QDQ_OK;
  const size_t rb = size_t(rows) * 4;
  const Span in[2] = {span(logits, rows, row_stride, n, eb), {tokens, rb}};
  const Span o[5] = {{logprob, rb}, {entropy, rb}, {k ? top_index : nullptr, rb * k}, {k ? top_logprob : nullptr, rb * k},
                     {workspace, workspace_bytes}};
  for (int i = 0; i < 5; ++i) {
    for (const Span &p : in)
      if (clash(o[i], p)) return QDQ_ERR_ALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (clash(o[i], o[j])) return QDQ_ERR_ALIAS;
  }
  if (workspace_bytes < token_logprobs_workspace_bytes(rows, n, k)) return QDQ_ERR_SCRATCH;
  return launch_token_logprobs(logits, row_stride, type, tokens, rows, n, k, workspace, workspace_bytes, logprob, entropy, top_index,
                               top_logprob, stream);
}

int qdq_kv_tree_attention(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                          int table_stride, const int *kv_len, const int *cu_q, const int *parent, int n_seqs, int max_q,
                          int max_kv_len, int n_heads, const void *q, long long q_stride, void *out, long long out_stride,
                          float *lse, const float *slopes, float scale, float softcap, int window, int type,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (n_seqs != 0 && max_q != 0 && (!cu_q || !parent)) return QDQ_ERR_NULL;
  if (max_q > QDQ_MAX_TREE) return QDQ_ERR_UNSUPPORTED;
  if (n_seqs == 0 || max_q == 0) cu_q = reinterpret_cast<const int *>(uintptr_t(256));  // (any; checked without being read)
  return attention(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, kv_len, cu_q, parent, n_seqs, max_q,
                   max_kv_len, n_heads, q, q_stride, out, out_stride, lse, slopes, scale, softcap, window, type, workspace,
                   workspace_bytes, stream);
}

int qdq_kv_append_rope(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                       int table_stride, const int *kv_len, const int *cu_new, const int *parent, int n_seqs, int max_new,
                       int n_heads, const void *q, long long q_stride, void *q_out, long long q_out_stride, const void *k,
                       long long k_stride, const void *v, long long v_stride, const float *q_weight,
                       const float *k_weight, float eps, const float *freqs, int n_rot, int interleaved, int type,
                       cudaStream_t stream) {
  const bool nothing = n_seqs == 0 || max_new == 0;
  if (!nothing && (!kv_len || !k || !v || (n_heads > 0 && (!q || !q_out)))) return QDQ_ERR_NULL;
  int rc = check_pool(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, n_seqs, nothing);
  if (rc != QDQ_OK) return rc;
  if (!type_ok(type) || max_new < 0 || (!cu_new && max_new != 1) || n_heads < 0 || !(eps >= 0.f)) return QDQ_ERR_DIMS;
  if (freqs && (n_rot < 8 || n_rot % 8 || n_rot > head_dim || (interleaved != 0 && interleaved != 1))) return QDQ_ERR_DIMS;
  if ((parent && max_new > QDQ_MAX_TREE) || n_heads > (1 << 20)) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(kv_len, 4) || !aligned(cu_new, 4) || !aligned(parent, 4) || !aligned(freqs, 4) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16))
    return QDQ_ERR_ALIGN;
  const int64_t width = int64_t(n_kv) * head_dim, q_width = int64_t(n_heads) * head_dim;
  if ((rc = check_rows(k, k_stride, width, type)) != QDQ_OK || (rc = check_rows(v, v_stride, width, type)) != QDQ_OK) return rc;
  if (n_heads > 0 && ((rc = check_rows(q, q_stride, q_width, type)) != QDQ_OK ||
                      (rc = check_rows(q_out, q_out_stride, q_width, type)) != QDQ_OK))
    return rc;
  if (nothing) return QDQ_OK;
  const int64_t known = cu_new ? 1 : n_seqs;  // new rows the host can count on
  const int eb = type_bytes(type);
  const Span sp{pages, size_t(n_pages) * page_bytes(page_tokens, n_kv, head_dim)};
  const Span sq = span(n_heads ? q : nullptr, known, q_stride, q_width, eb), so = span(n_heads ? q_out : nullptr, known, q_out_stride, q_width, eb);
  const Span in[9] = {span(k, known, k_stride, width, eb),
                      span(v, known, v_stride, width, eb),
                      {page_table, size_t(n_seqs) * table_stride * 4},
                      {kv_len, size_t(n_seqs) * 4},
                      {cu_new, size_t(n_seqs + 1) * 4},
                      {parent, size_t(known) * 4},
                      {q_weight, size_t(head_dim) * 4},
                      {k_weight, size_t(head_dim) * 4},
                      {freqs, freqs ? size_t(n_rot / 2) * 4 : 0}};
  for (const Span &i : in)
    if (clash(i, sp) || clash(i, so)) return QDQ_ERR_ALIAS;
  if (clash(sp, sq) || clash(sp, so) || (clash(so, sq) && !(q_out == q && q_out_stride == q_stride))) return QDQ_ERR_ALIAS;
  const KvPool c{static_cast<uint8_t *>(pages), page_table, n_pages, page_tokens, n_kv, table_stride};
  return launch_kv_append_rope(c, head_dim, kv_len, cu_new, parent, n_seqs, max_new, n_heads, q, q_stride, q_out, q_out_stride, k,
                               k_stride, v, v_stride, q_weight, k_weight, eps, freqs, n_rot, interleaved, type, stream);
}

int qdq_kv_keep(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table, int table_stride,
                const int *kv_len, const int *cu, int n_seqs, const int *path, int path_stride, const int *accepted,
                cudaStream_t stream) {
  const bool nothing = n_seqs == 0;
  if (!nothing && (!kv_len || !cu || !path || !accepted)) return QDQ_ERR_NULL;
  const int rc = check_pool(pages, n_pages, page_tokens, n_kv, head_dim, page_table, table_stride, n_seqs, nothing);
  if (rc != QDQ_OK) return rc;
  if (path_stride < 1) return QDQ_ERR_DIMS;
  if (!aligned(kv_len, 4) || !aligned(cu, 4) || !aligned(path, 4) || !aligned(accepted, 4)) return QDQ_ERR_ALIGN;
  if (nothing) return QDQ_OK;
  const Span sp{pages, size_t(n_pages) * page_bytes(page_tokens, n_kv, head_dim)};
  const Span in[5] = {{page_table, size_t(n_seqs) * table_stride * 4},
                      {kv_len, size_t(n_seqs) * 4},
                      {cu, size_t(n_seqs + 1) * 4},
                      {path, size_t(n_seqs) * path_stride * 4},
                      {accepted, size_t(n_seqs) * 4}};
  for (const Span &i : in)
    if (clash(i, sp)) return QDQ_ERR_ALIAS;
  const KvPool c{static_cast<uint8_t *>(pages), page_table, n_pages, page_tokens, n_kv, table_stride};
  return launch_kv_keep(c, head_dim, kv_len, cu, n_seqs, path, path_stride, accepted, stream);
}

size_t qdq_verify_drafts_workspace_bytes(int n_seqs, int max_rows, int n) {
  if (n_seqs < 1 || max_rows < 1 || max_rows > QDQ_MAX_TREE || n < 1 || n > (1 << 30)) return 0;
  return verify_drafts_workspace_bytes(n_seqs, max_rows, n);
}

int qdq_verify_drafts(const void *logits, long long row_stride, int type, const int *tokens, const int *cu, const int *parent,
                      int n_seqs, int max_rows, int n, const float *draft_probs, long long draft_stride,
                      const float *uniform, float temperature, int *accepted, int *path, int *next_token, void *workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  const bool nothing = n_seqs == 0;
  if (!nothing && (!logits || !accepted || !path || !next_token || !workspace || (!tokens && max_rows > 1) ||
                   (!uniform && temperature != 0.f)))
    return QDQ_ERR_NULL;
  if (!type_ok(type) || n_seqs < 0 || max_rows < 1 || (!cu && max_rows != 1) || n < 1 || row_stride < n ||
      (draft_probs && draft_stride < n) || !(temperature == 0.f || (temperature >= 1e-6f && temperature <= 1e6f)))
    return QDQ_ERR_DIMS;
  if (max_rows > QDQ_MAX_TREE || n > (1 << 30)) return QDQ_ERR_UNSUPPORTED;
  const int eb = type_bytes(type);
  if (!aligned(logits, eb) || !aligned(tokens, 4) || !aligned(cu, 4) || !aligned(parent, 4) || !aligned(draft_probs, 4) ||
      !aligned(uniform, 4) || !aligned(accepted, 4) || !aligned(path, 4) || !aligned(next_token, 4) || !aligned(workspace, 256))
    return QDQ_ERR_ALIGN;
  if (nothing) return QDQ_OK;
  const int64_t known = cu ? 1 : n_seqs;  // rows the host can count on
  const size_t rb = size_t(known) * 4, sb = size_t(n_seqs) * 4;
  const Span in[6] = {span(logits, known, row_stride, n, eb), span(draft_probs, known, draft_stride, n, 4), {tokens, rb},
                      {cu, sb + 4}, {parent, rb}, {uniform, rb}};
  const Span o[4] = {{accepted, sb}, {path, sb * max_rows}, {next_token, sb}, {workspace, workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Span &p : in)
      if (clash(o[i], p)) return QDQ_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (clash(o[i], o[j])) return QDQ_ERR_ALIAS;
  }
  if (workspace_bytes < verify_drafts_workspace_bytes(n_seqs, max_rows, n)) return QDQ_ERR_SCRATCH;
  return launch_verify_drafts(logits, row_stride, type, tokens, cu, parent, n_seqs, max_rows, n, draft_probs, draft_stride, uniform,
                              temperature, accepted, path, next_token, workspace, workspace_bytes, stream);
}

}  // extern "C"

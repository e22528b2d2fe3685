// Argument marshalling of the decode-step operators in C: what the Python binding does for the
// ordinary case (tensors of the right types, packed), without the interpreter's share of a call
// (a one-row norm: 8 us through ctypes, of which 2 are the launch).  Anything unusual -- another
// type, a stride, a wrong shape, too few elements -- is left to the Python code, which names the error: the
// functions then return None.  Only the Python C API is used; tensors are read through their
// Python attributes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "qdq.h"

namespace {

PyObject *s_dtype, *s_shape, *s_contig, *s_ptr, *s_nbytes, *s_numel, *s_cuda;
PyObject *g_types[3], *g_int32;  // torch.float32, float16, bfloat16; torch.int32
decltype(&qdq_rms_norm) f_norm;
decltype(&qdq_kv_append) f_append;
decltype(&qdq_kv_read) f_read;
decltype(&qdq_kv_attention) f_attention;
decltype(&qdq_token_logprobs) f_logprobs;
decltype(&qdq_kv_append_rope) f_rope;
decltype(&qdq_kv_tree_attention) f_tree;
decltype(&qdq_verify_drafts) f_verify;
decltype(&qdq_kv_keep) f_keep;

// Reads arguments; `ok` falls to false at the first one that is not ordinary.
struct Reader {
  bool ok = true;

  PyObject *attr(PyObject *o, PyObject *name) {  // a new reference or NULL
    PyObject *r = ok ? PyObject_GetAttr(o, name) : nullptr;
    if (!r) ok = false;
    return r;
  }
  bool is(PyObject *o, PyObject *name, PyObject *want) {
    PyObject *r = attr(o, name);
    const bool same = r == want;
    Py_XDECREF(r);
    return same;
  }
  long long integer(PyObject *o) {
    if (!ok) return 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  int small(PyObject *o) {
    const long long v = integer(o);
    if (v < -0x7fffffffll || v > 0x7fffffffll) ok = false;
    return int(v);
  }
  double real(PyObject *o) {
    if (!ok) return 0;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return v;
  }
  void *address(PyObject *o) {  // of a CUDA tensor; NULL for None
    if (!ok || o == Py_None) return nullptr;
    if (!is(o, s_cuda, Py_True)) {
      ok = false;
      return nullptr;
    }
    PyObject *r = PyObject_CallMethodNoArgs(o, s_ptr);
    void *p = nullptr;
    if (r) {
      p = PyLong_AsVoidPtr(r);
      Py_DECREF(r);
    }
    if (!r || PyErr_Occurred()) ok = false;
    return p;
  }
  void contiguous(PyObject *o) {
    PyObject *r = ok ? PyObject_CallMethodNoArgs(o, s_contig) : nullptr;
    if (r != Py_True) ok = false;
    Py_XDECREF(r);
  }
  int type(PyObject *o) {
    PyObject *r = attr(o, s_dtype);
    int t = 0;
    while (t < 3 && r != g_types[t]) ++t;
    if (t == 3) ok = false;
    Py_XDECREF(r);
    return t;
  }
  // Address of a packed tensor of one element type; NULL for None.
  void *packed(PyObject *o, PyObject *dtype) {
    if (!ok || o == Py_None) return nullptr;
    if (!is(o, s_dtype, dtype)) ok = false;
    contiguous(o);
    return address(o);
  }
  // ... of at least `least` elements.
  void *vec(PyObject *o, PyObject *dtype, long long least) {
    if (!ok || o == Py_None) return nullptr;
    PyObject *r = PyObject_CallMethodNoArgs(o, s_numel);
    if (!r || integer(r) < least) ok = false;
    Py_XDECREF(r);
    return packed(o, dtype);
  }
  // ... whose first dimension is at least `least` rows of `width` elements.
  void *rows(PyObject *o, long long width, PyObject *dtype, long long *stride, long long least) {
    *stride = 0;
    if (!ok || o == Py_None) return nullptr;
    PyObject *shape = attr(o, s_shape);
    long long w = 1;
    if (!shape || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) < 2) ok = false;
    if (ok && integer(PyTuple_GET_ITEM(shape, 0)) < least) ok = false;
    for (Py_ssize_t i = 1; ok && i < PyTuple_GET_SIZE(shape); ++i) w *= integer(PyTuple_GET_ITEM(shape, i));
    Py_XDECREF(shape);
    if (w != width) ok = false;
    *stride = width;
    return packed(o, dtype);
  }
  // Address of a packed tensor of at least `least` bytes; NULL for None.
  void *bytes(PyObject *o, long long least, size_t *size) {
    *size = 0;
    if (!ok || o == Py_None) return nullptr;
    *size = nbytes(o);
    if (ok && (long long)*size < least) ok = false;
    contiguous(o);
    return address(o);
  }
  size_t nbytes(PyObject *o) {
    PyObject *r = attr(o, s_nbytes);
    const long long v = r ? integer(r) : 0;
    Py_XDECREF(r);
    return size_t(v);
  }
};

// The pool and its table: pages, page_table, n_kv, head_dim, page_tokens.
struct Pool {
  void *pages;
  const int *table;
  int n_pages, page_tokens, n_kv, head_dim, seqs, width;
  Pool(Reader &r, PyObject *p, PyObject *t, PyObject *kv, PyObject *dim, PyObject *page) {
    n_kv = r.small(kv);
    head_dim = r.small(dim);
    page_tokens = r.small(page);
    const long long rec = (2ll * page_tokens * head_dim + page_tokens / 2 + 127) / 128 * 128 * n_kv;
    const long long all = (long long)r.nbytes(p);
    if (rec <= 0 || all % rec || all / rec > 0x7fffffff) r.ok = false;
    n_pages = r.ok ? int(all / rec) : 0;
    r.contiguous(p);
    pages = r.address(p);
    PyObject *shape = r.attr(t, s_shape);
    if (!shape || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != 2) r.ok = false;
    seqs = r.ok ? r.small(PyTuple_GET_ITEM(shape, 0)) : 0;
    width = r.ok ? r.small(PyTuple_GET_ITEM(shape, 1)) : 0;
    Py_XDECREF(shape);
    table = static_cast<const int *>(r.packed(t, g_int32));
  }
};

PyObject *leave() {  // to the Python code
  PyErr_Clear();
  Py_RETURN_NONE;
}
cudaStream_t stream_of(Reader &r, PyObject *o) { return o == Py_None ? nullptr : reinterpret_cast<cudaStream_t>(r.integer(o)); }

// x, weight, out, rows, n, eps, residual, sum_out, q8_out, stream
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 10 || !f_norm) return leave();
  const int t = r.type(a[0]), rows = r.small(a[3]), n = r.small(a[4]);
  if (!r.ok) return leave();
  long long xs, rs, ss, os;
  void *x = r.rows(a[0], n, g_types[t], &xs, rows), *res = r.rows(a[6], n, g_types[t], &rs, rows);
  void *sum = r.rows(a[7], n, g_types[t], &ss, rows), *out = r.rows(a[2], n, g_types[t], &os, rows);
  const float *w = static_cast<const float *>(r.vec(a[1], g_types[0], n));
  size_t qb;
  void *q8 = r.bytes(a[8], (long long)rows * (n / 32) * 34, &qb);
  const float eps = float(r.real(a[5]));
  const cudaStream_t st = stream_of(r, a[9]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_norm(x, res, w, sum, out, q8, t, rows, n, xs, rs, ss, os, eps, st));
}

// pages, table, kv_len, k, v, n_kv, head_dim, page_tokens, cu_new, max_new, stream
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 11 || !f_append) return leave();
  const Pool p(r, a[0], a[1], a[5], a[6], a[7]);
  const int t = r.type(a[3]);
  if (!r.ok) return leave();
  long long ks, vs;
  const int *len = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[8], g_int32, p.seqs + 1ll));
  const long long wide = (long long)p.n_kv * p.head_dim, least = cu ? 0 : p.seqs;
  void *k = r.rows(a[3], wide, g_types[t], &ks, least), *v = r.rows(a[4], wide, g_types[t], &vs, least);
  const int most = r.small(a[9]);
  const cudaStream_t st = stream_of(r, a[10]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_append(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, len, cu, p.seqs, most, k, v, ks,
                                  vs, t, st));
}

// pages, table, start, cu, k, v, n_kv, head_dim, page_tokens, max_tokens, stream
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 11 || !f_read) return leave();
  const Pool p(r, a[0], a[1], a[6], a[7], a[8]);
  const int t = r.type(a[4]);
  if (!r.ok) return leave();
  long long ks, vs;
  const int *start = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[3], g_int32, p.seqs + 1ll));
  const long long wide = (long long)p.n_kv * p.head_dim;
  void *k = r.rows(a[4], wide, g_types[t], &ks, 0), *v = r.rows(a[5], wide, g_types[t], &vs, 0);
  const int most = r.small(a[9]);
  const cudaStream_t st = stream_of(r, a[10]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_read(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, start, cu, p.seqs, most, k, v, ks,
                                vs, t, st));
}

// pages, table, kv_len, q, out, workspace, n_heads, n_kv, head_dim, page_tokens, max_kv_len, cu_q, max_q, scale, softcap,
// window, slopes, lse, stream
PyObject *kv_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 19 || !f_attention) return leave();
  const Pool p(r, a[0], a[1], a[7], a[8], a[9]);
  const int t = r.type(a[3]), heads = r.small(a[6]);
  if (!r.ok) return leave();
  long long qs, os;
  const int *len = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[11], g_int32, p.seqs + 1ll));
  const long long wide = (long long)heads * p.head_dim, least = cu ? 0 : p.seqs;
  void *q = r.rows(a[3], wide, g_types[t], &qs, least), *out = r.rows(a[4], wide, g_types[t], &os, least);
  size_t wb;
  void *ws = r.bytes(a[5], 0, &wb);
  const int most_kv = r.small(a[10]), most_q = r.small(a[12]), window = r.small(a[15]);
  const float scale = float(r.real(a[13])), cap = float(r.real(a[14]));
  const float *slopes = static_cast<const float *>(r.vec(a[16], g_types[0], heads));
  float *lse = static_cast<float *>(r.vec(a[17], g_types[0], least * heads));
  const cudaStream_t st = stream_of(r, a[18]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_attention(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, len, cu, p.seqs, most_q,
                                     most_kv, heads, q, qs, out, os, lse, slopes, scale, cap, window, t, ws, wb, st));
}

// logits, tokens, logprob, entropy, rows, n, workspace, k, top_index, top_logprob, stream
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 11 || !f_logprobs) return leave();
  const int t = r.type(a[0]), rows = r.small(a[4]), n = r.small(a[5]), k = r.small(a[7]);
  if (!r.ok) return leave();
  long long xs;
  void *x = r.rows(a[0], n, g_types[t], &xs, rows);
  const int *tokens = static_cast<const int *>(r.vec(a[1], g_int32, rows));
  float *lp = static_cast<float *>(r.vec(a[2], g_types[0], rows)), *ent = static_cast<float *>(r.vec(a[3], g_types[0], rows));
  int *ti = static_cast<int *>(r.vec(a[8], g_int32, (long long)rows * k));
  float *tl = static_cast<float *>(r.vec(a[9], g_types[0], (long long)rows * k));
  size_t wb;
  void *ws = r.bytes(a[6], 0, &wb);
  const cudaStream_t st = stream_of(r, a[10]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_logprobs(x, xs, t, tokens, rows, n, k, lp, ent, ti, tl, ws, wb, st));
}

// pages, table, kv_len, q, q_out, k, v, n_heads, n_kv, head_dim, page_tokens, freqs, interleaved, q_weight, k_weight, eps, cu_new,
// max_new, parent, stream
PyObject *kv_append_rope(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 20 || !f_rope) return leave();
  const Pool p(r, a[0], a[1], a[8], a[9], a[10]);
  const int t = r.type(a[5]), heads = r.small(a[7]);
  if (!r.ok) return leave();
  long long qs, os, ks, vs;
  const int *len = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[16], g_int32, p.seqs + 1ll));
  const long long wide = (long long)p.n_kv * p.head_dim, q_wide = (long long)heads * p.head_dim, least = cu ? 0 : p.seqs;
  void *q = r.rows(a[3], q_wide, g_types[t], &qs, least), *o = r.rows(a[4], q_wide, g_types[t], &os, least);
  void *k = r.rows(a[5], wide, g_types[t], &ks, least), *v = r.rows(a[6], wide, g_types[t], &vs, least);
  int n_rot = 0;
  if (r.ok && a[11] != Py_None) {
    PyObject *n = PyObject_CallMethodNoArgs(a[11], s_numel);
    if (n) {
      n_rot = 2 * r.small(n);
      Py_DECREF(n);
    } else {
      r.ok = false;
    }
  }
  const float *freqs = static_cast<const float *>(r.vec(a[11], g_types[0], 0));
  const int pairs = r.ok ? PyObject_IsTrue(a[12]) : 0, most = r.small(a[17]);
  if (pairs < 0) r.ok = false;
  const float *qw = static_cast<const float *>(r.vec(a[13], g_types[0], p.head_dim)), *kw = static_cast<const float *>(r.vec(a[14], g_types[0], p.head_dim));
  const float eps = float(r.real(a[15]));
  const int *parent = static_cast<const int *>(r.vec(a[18], g_int32, least));
  const cudaStream_t st = stream_of(r, a[19]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_rope(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, len, cu, parent, p.seqs, most, heads,
                                q, qs, o, os, k, ks, v, vs, qw, kw, eps, freqs, n_rot, pairs, t, st));
}

// pages, table, kv_len, q, out, workspace, n_heads, n_kv, head_dim, page_tokens, max_kv_len, cu_q, max_q, scale, softcap,
// window, slopes, lse, parent, stream
PyObject *kv_tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 20 || !f_tree) return leave();
  const Pool p(r, a[0], a[1], a[7], a[8], a[9]);
  const int t = r.type(a[3]), heads = r.small(a[6]);
  if (!r.ok) return leave();
  long long qs, os;
  const int *len = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[11], g_int32, p.seqs + 1ll));
  const long long wide = (long long)heads * p.head_dim;
  void *q = r.rows(a[3], wide, g_types[t], &qs, 0), *out = r.rows(a[4], wide, g_types[t], &os, 0);
  size_t wb;
  void *ws = r.bytes(a[5], 0, &wb);
  const int most_kv = r.small(a[10]), most_q = r.small(a[12]), window = r.small(a[15]);
  const float scale = float(r.real(a[13])), cap = float(r.real(a[14]));
  const float *slopes = static_cast<const float *>(r.vec(a[16], g_types[0], heads));
  float *lse = static_cast<float *>(r.vec(a[17], g_types[0], 0));
  const int *parent = static_cast<const int *>(r.vec(a[18], g_int32, 0));
  const cudaStream_t st = stream_of(r, a[19]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_tree(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, len, cu, parent, p.seqs, most_q,
                                most_kv, heads, q, qs, out, os, lse, slopes, scale, cap, window, t, ws, wb, st));
}

// logits, tokens, uniform, accepted, path, next_token, n, workspace, cu, max_rows, parent, draft_probs, temperature, stream
PyObject *verify_drafts(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 14 || !f_verify) return leave();
  const int t = r.type(a[0]), n = r.small(a[6]), rows = r.small(a[9]);
  PyObject *count = r.ok ? PyObject_CallMethodNoArgs(a[3], s_numel) : nullptr;
  const int seqs = count ? r.small(count) : 0;
  Py_XDECREF(count);
  if (!r.ok || !count) return leave();
  const int *cu = static_cast<const int *>(r.vec(a[8], g_int32, seqs + 1ll));
  const long long least = cu ? 0 : seqs;
  long long xs, ds;
  void *x = r.rows(a[0], n, g_types[t], &xs, least);
  const float *probs = static_cast<const float *>(r.rows(a[11], n, g_types[0], &ds, least));
  const int *tokens = static_cast<const int *>(r.vec(a[1], g_int32, least)), *parent = static_cast<const int *>(r.vec(a[10], g_int32, least));
  const float *uniform = static_cast<const float *>(r.vec(a[2], g_types[0], least));
  int *accepted = static_cast<int *>(r.vec(a[3], g_int32, 0)), *path = static_cast<int *>(r.vec(a[4], g_int32, (long long)seqs * rows));
  int *next = static_cast<int *>(r.vec(a[5], g_int32, seqs));
  size_t wb;
  void *ws = r.bytes(a[7], 0, &wb);
  const float temperature = float(r.real(a[12]));
  const cudaStream_t st = stream_of(r, a[13]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_verify(x, xs, t, tokens, cu, parent, seqs, rows, n, probs, ds, uniform, temperature, accepted, path, next, ws, wb,
                                  st));
}

// pages, table, kv_len, cu, path, accepted, n_kv, head_dim, page_tokens, stream
PyObject *kv_keep(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  Reader r;
  if (n_args != 10 || !f_keep) return leave();
  const Pool p(r, a[0], a[1], a[6], a[7], a[8]);
  if (!r.ok) return leave();
  const int *len = static_cast<const int *>(r.vec(a[2], g_int32, p.seqs)), *cu = static_cast<const int *>(r.vec(a[3], g_int32, p.seqs + 1ll));
  PyObject *shape = r.attr(a[4], s_shape);
  if (!shape || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != 2 || r.integer(PyTuple_GET_ITEM(shape, 0)) < p.seqs) r.ok = false;
  const int width = r.ok ? r.small(PyTuple_GET_ITEM(shape, 1)) : 0;
  Py_XDECREF(shape);
  const int *path = static_cast<const int *>(r.vec(a[4], g_int32, 0)), *accepted = static_cast<const int *>(r.vec(a[5], g_int32, p.seqs));
  const cudaStream_t st = stream_of(r, a[9]);
  if (!r.ok) return leave();
  return PyLong_FromLong(f_keep(p.pages, p.n_pages, p.page_tokens, p.n_kv, p.head_dim, p.table, p.width, len, cu, p.seqs, path, width, accepted,
                                st));
}

// Addresses of the nine functions in the loaded library, then torch.float32, float16, bfloat16, int32.
constexpr int kFunctions = 9;
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  if (n_args != kFunctions + 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes 13 arguments");
    return nullptr;
  }
  void *f[kFunctions];
  for (int i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_norm = reinterpret_cast<decltype(f_norm)>(f[0]);
  f_append = reinterpret_cast<decltype(f_append)>(f[1]);
  f_read = reinterpret_cast<decltype(f_read)>(f[2]);
  f_attention = reinterpret_cast<decltype(f_attention)>(f[3]);
  f_logprobs = reinterpret_cast<decltype(f_logprobs)>(f[4]);
  f_rope = reinterpret_cast<decltype(f_rope)>(f[5]);
  f_tree = reinterpret_cast<decltype(f_tree)>(f[6]);
  f_verify = reinterpret_cast<decltype(f_verify)>(f[7]);
  f_keep = reinterpret_cast<decltype(f_keep)>(f[8]);
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[kFunctions + i]);
    Py_XSETREF(g_types[i], a[kFunctions + i]);
  }
  Py_INCREF(a[kFunctions + 3]);
  Py_XSETREF(g_int32, a[kFunctions + 3]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),         FAST(rms_norm),       FAST(kv_append), FAST(kv_read),
                         FAST(kv_attention), FAST(token_logprobs), FAST(kv_append_rope), FAST(kv_tree_attention),
                         FAST(verify_drafts), FAST(kv_keep), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_contig = PyUnicode_InternFromString("is_contiguous");
  s_ptr = PyUnicode_InternFromString("data_ptr");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  s_numel = PyUnicode_InternFromString("numel");
  s_cuda = PyUnicode_InternFromString("is_cuda");
  return PyModule_Create(&module);
}

/* decode_py.c -- the Python side of the decode-step entry points, as an
 * extension module over libprism.so's C ABI (include/prism.h): reads the
 * tensors' addresses, shapes and strides, checks them, allocates outputs and
 * workspaces through torch.empty, and calls.
 *
 * A decode step is a chain of kernels of 5 to 20 us, so the host time of a call
 * is part of its cost: a 4-bit linear call takes CALLNEW us here against CALLOLD us of
 * the same checks in Python with ctypes.  Only Python's own C API is used: what is
 * asked of a tensor are its public attributes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "prism.h"

/* What setup() hands over. */
static PyObject *g_tensor, *g_bf16, *g_f16, *g_f32, *g_i8, *g_u8, *g_i32, *g_empty, *g_raw_stream, *g_check;
static PyObject *s_dtype, *s_shape, *s_device, *s_stride, *s_data_ptr, *s_get_device, *s_cuda_stream, *s_empty_kw;

#define MAX_RANK 4

typedef struct {
  void *ptr;
  int rank;
  int64_t shape[MAX_RANK], stride[MAX_RANK];
} Operand;

static int is_tensor(PyObject *t, const char *name) {
  if (PyObject_TypeCheck(t, (PyTypeObject *)g_tensor)) return 1;
  PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return 0;
}

/* A tuple of integers; its length, or -1. */
static int read_ints(PyObject *tuple, int64_t *out) {
  int n = -1;
  if (tuple != NULL && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) <= MAX_RANK) {
    n = (int)PyTuple_GET_SIZE(tuple);
    for (int i = 0; i < n; ++i) {
      out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
      if (out[i] == -1 && PyErr_Occurred()) {
        n = -1;
        break;
      }
    }
  }
  Py_XDECREF(tuple);
  return n;
}

static int device_of(PyObject *t, int64_t *device) {
  PyObject *d = PyObject_CallMethodNoArgs(t, s_get_device);
  if (d == NULL) return 0;
  *device = PyLong_AsLongLong(d);
  Py_DECREF(d);
  return *device != -1 || !PyErr_Occurred();
}

/* The CUDA device index of the first operand, with its shape of n dimensions. */
static int first_operand(PyObject *t, const char *name, int n, int64_t *device, Operand *o) {
  if (!is_tensor(t, name)) return 0;
  if (!device_of(t, device)) return 0;
  if (*device < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be on a CUDA device", name);
    return 0;
  }
  o->rank = read_ints(PyObject_GetAttr(t, s_shape), o->shape);
  if (o->rank != n) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s must have %d dims", name, n);
    return 0;
  }
  return 1;
}

/* Only the shape, of n dimensions. */
static int shape_of(PyObject *t, const char *name, int n, int64_t *shape) {
  int64_t read[MAX_RANK];
  if (!is_tensor(t, name)) return 0;
  if (read_ints(PyObject_GetAttr(t, s_shape), read) != n) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s must have %d dims", name, n);
    return 0;
  }
  for (int i = 0; i < n; ++i) shape[i] = read[i];
  return 1;
}

/* A tensor of this dtype and shape on this device, its last dimension
 * contiguous (dense: all of them). */
static int operand(PyObject *t, const char *name, PyObject *dtype, int64_t device, int n, const int64_t *shape, int dense,
                   Operand *o) {
  if (!is_tensor(t, name)) return 0;
  PyObject *have = PyObject_GetAttr(t, s_dtype);
  if (have == NULL) return 0;
  const int same = have == dtype;
  if (!same) PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, have);
  Py_DECREF(have);
  if (!same) return 0;
  int64_t on;
  if (!device_of(t, &on)) return 0;
  if (on != device) {
    PyErr_Format(PyExc_ValueError, "%s must be on cuda:%lld, got device index %lld", name, (long long)device, (long long)on);
    return 0;
  }
  o->rank = read_ints(PyObject_GetAttr(t, s_shape), o->shape);
  int fits = o->rank == n;
  for (int i = 0; fits && i < n; ++i) fits = o->shape[i] == shape[i];
  if (!fits) {
    if (PyErr_Occurred()) return 0;
    char want[128];
    int at = 0;
    for (int i = 0; i < n; ++i) at += snprintf(want + at, sizeof want - at, i ? ", %lld" : "%lld", (long long)shape[i]);
    PyObject *got = PyObject_GetAttr(t, s_shape);
    if (got == NULL) return 0;
    PyErr_Format(PyExc_ValueError, "%s must be of shape [%s], got %S", name, want, got);
    Py_DECREF(got);
    return 0;
  }
  if (read_ints(PyObject_CallMethodNoArgs(t, s_stride), o->stride) != n) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s must have %d strides", name, n);
    return 0;
  }
  if (o->stride[n - 1] != 1 && shape[n - 1] > 1) {
    PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
    return 0;
  }
  if (dense) {
    int64_t step = 1, numel = 1;
    for (int i = 0; i < n; ++i) numel *= shape[i];
    for (int i = n - 1; numel > 0 && i >= 0; --i) {
      if (shape[i] != 1 && o->stride[i] != step) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
        return 0;
      }
      step *= shape[i];
    }
  }
  PyObject *p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (p == NULL) return 0;
  o->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

/* The address of an optional dense operand, NULL for None. */
static int optional(PyObject *t, const char *name, PyObject *dtype, int64_t device, int n, const int64_t *shape, void **ptr) {
  Operand o;
  *ptr = NULL;
  if (t == Py_None) return 1;
  if (!operand(t, name, dtype, device, n, shape, 1, &o)) return 0;
  *ptr = o.ptr;
  return 1;
}

/* torch.empty of this shape on the device of `like`; its address. */
static PyObject *empty(PyObject *like, PyObject *dtype, int n, const int64_t *shape, void **ptr) {
  PyObject *out = NULL, *p, *device = PyObject_GetAttr(like, s_device), *size = PyTuple_New(n);
  if (device != NULL && size != NULL) {
    int ok = 1;
    for (int i = 0; i < n; ++i) {
      PyObject *v = PyLong_FromLongLong(shape[i]);
      if (v == NULL) ok = 0;
      PyTuple_SET_ITEM(size, i, v);
    }
    PyObject *args[3] = {size, dtype, device};
    if (ok) out = PyObject_Vectorcall(g_empty, args, 1, s_empty_kw);
  }
  Py_XDECREF(device);
  Py_XDECREF(size);
  if (out == NULL) return NULL;
  p = PyObject_CallMethodNoArgs(out, s_data_ptr);
  if (p == NULL) {
    Py_DECREF(out);
    return NULL;
  }
  *ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return out;
}

static int stream_of(PyObject *stream, int64_t device, void **out) {
  PyObject *v;
  if (stream == Py_None) {
    PyObject *d = PyLong_FromLongLong(device);
    if (d == NULL) return 0;
    v = PyObject_CallOneArg(g_raw_stream, d);
    Py_DECREF(d);
  } else {
    v = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (v == NULL) return 0;
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

static int integer(PyObject *v, int64_t *out) {
  *out = PyLong_AsLongLong(v);
  return *out != -1 || !PyErr_Occurred();
}

/* None, or the exception for a status that is not PRISM_OK. */
static PyObject *answer(const char *fn, int status) {
  if (status == PRISM_OK) Py_RETURN_NONE;
  return PyObject_CallFunction(g_check, "si", fn, status);
}

static int argc_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
  return 0;
}

/* The cache's own tensors: its geometry and the addresses of codes, scales,
 * page table and lengths. */
typedef struct {
  int64_t num_pages, heads, block, d, seqs, max_pages, ld_table;
  void *k_codes, *v_codes, *k_scale, *v_scale, *table, *lens;
} Cache;

static int read_cache(PyObject *seq, PyObject *page_table, PyObject *seq_lens, int64_t device, Cache *c) {
  PyObject **t = PySequence_Fast_ITEMS(seq);
  if (PySequence_Fast_GET_SIZE(seq) < 4) {
    PyErr_SetString(PyExc_ValueError, "cache must have k_codes, v_codes, k_scale, v_scale");
    return 0;
  }
  int64_t shape[4], table_shape[2];
  Operand o;
  if (!shape_of(t[0], "k_codes", 4, shape) || !shape_of(page_table, "page_table", 2, table_shape)) return 0;
  c->num_pages = shape[0], c->heads = shape[1], c->block = shape[2], c->d = shape[3];
  c->seqs = table_shape[0], c->max_pages = table_shape[1];
  if (!operand(t[0], "k_codes", g_i8, device, 4, shape, 1, &o)) return 0;
  c->k_codes = o.ptr;
  if (!operand(t[1], "v_codes", g_i8, device, 4, shape, 1, &o)) return 0;
  c->v_codes = o.ptr;
  if (!operand(t[2], "k_scale", g_f32, device, 2, shape, 1, &o)) return 0;
  c->k_scale = o.ptr;
  if (!operand(t[3], "v_scale", g_f32, device, 2, shape, 1, &o)) return 0;
  c->v_scale = o.ptr;
  if (!operand(page_table, "page_table", g_i32, device, 2, table_shape, 0, &o)) return 0;
  c->table = o.ptr, c->ld_table = o.stride[0];
  if (!operand(seq_lens, "seq_lens", g_i32, device, 1, table_shape, 0, &o)) return 0;
  c->lens = o.ptr;
  return 1;
}

static int offsets(PyObject *cu, const char *name, int64_t seqs, int64_t rows, int64_t device, void **ptr) {
  const int64_t n = seqs + 1;
  Operand o;
  *ptr = NULL;
  if (cu != Py_None) {
    if (!operand(cu, name, g_i32, device, 1, &n, 0, &o)) return 0;
    *ptr = o.ptr;
  } else if (rows != seqs) {
    PyErr_Format(PyExc_ValueError, "without %s there is one row for each sequence", name);
    return 0;
  }
  return 1;
}

/* A contiguous tensor of any type; its address and bytes. */
static int workspace(PyObject *t, int64_t device, void **ptr, int64_t *bytes) {
  int64_t on;
  if (!is_tensor(t, "workspace") || !device_of(t, &on)) return 0;
  PyObject *whole = PyObject_CallMethod(t, "is_contiguous", NULL), *p = PyObject_CallMethodNoArgs(t, s_data_ptr),
           *size = PyObject_GetAttrString(t, "nbytes");
  const int ok = whole != NULL && p != NULL && size != NULL;
  if (ok && (on != device || whole != Py_True))
    PyErr_Format(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:%lld", (long long)device);
  if (ok) {
    *ptr = PyLong_AsVoidPtr(p);
    *bytes = PyLong_AsLongLong(size);
  }
  Py_XDECREF(whole);
  Py_XDECREF(p);
  Py_XDECREF(size);
  return !PyErr_Occurred();
}

static const int64_t kOne = 1;

/* append(k, v, cache, page_table, seq_lens, cu_new, max_new, err, stream) */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (!argc_is(n, 9)) return NULL;
  int64_t device, max_new;
  Operand k, v, ko, vo;
  Cache c;
  void *cu, *err, *stream;
  if (!first_operand(a[0], "k", 3, &device, &k)) return NULL;
  PyObject *cache = PySequence_Fast(a[2], "cache must be a sequence of tensors"), *out = NULL;
  if (cache == NULL) return NULL;
  if (!read_cache(cache, a[3], a[4], device, &c)) goto done;
  if (PySequence_Fast_GET_SIZE(cache) < 6) {
    PyErr_SetString(PyExc_ValueError, "cache must have k_open and v_open");
    goto done;
  }
  const int64_t rows = k.shape[0], shape[3] = {rows, c.heads, c.d}, open[4] = {c.seqs, c.heads, c.block, c.d};
  if (!operand(a[0], "k", g_bf16, device, 3, shape, 0, &k) || !operand(a[1], "v", g_bf16, device, 3, shape, 0, &v) ||
      !operand(PySequence_Fast_GET_ITEM(cache, 4), "k_open", g_bf16, device, 4, open, 1, &ko) ||
      !operand(PySequence_Fast_GET_ITEM(cache, 5), "v_open", g_bf16, device, 4, open, 1, &vo) ||
      !offsets(a[5], "cu_new", c.seqs, rows, device, &cu))
    goto done;
  max_new = cu == NULL || rows < 1 ? 1 : rows;
  if (a[6] != Py_None && !integer(a[6], &max_new)) goto done;
  if (!optional(a[7], "err", g_i32, device, 1, &kOne, &err) || !stream_of(a[8], device, &stream)) goto done;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_kv_append(k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1], c.k_codes, c.v_codes,
                           c.k_scale, c.v_scale, ko.ptr, vo.ptr, c.table, c.ld_table, c.lens, cu, c.seqs, rows, max_new,
                           c.num_pages, c.max_pages, c.heads, c.d, c.block, err, stream);
  Py_END_ALLOW_THREADS
  out = answer("prism_kv_append", status);
done:
  Py_DECREF(cache);
  return out;
}

/* attention(q, cache, page_table, seq_lens, cu_q, max_q, scale, causal, window, out, lse, workspace, err, stream) */
static PyObject *py_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (!argc_is(n, 14)) return NULL;
  int64_t device, max_q, window, ws_bytes = 0;
  Operand q, o;
  Cache c;
  void *cu, *lse, *err, *stream, *ws = NULL;
  PyObject *out = NULL, *held = NULL;
  int done = 0;
  if (!first_operand(a[0], "q", 3, &device, &q)) return NULL;
  PyObject *cache = PySequence_Fast(a[1], "cache must be a sequence of tensors");
  if (cache == NULL) return NULL;
  if (!read_cache(cache, a[2], a[3], device, &c)) goto done;
  const int64_t rows = q.shape[0], heads = q.shape[1], shape[3] = {rows, heads, c.d};
  if (q.shape[2] != c.d || heads == 0 || c.heads == 0 || heads % c.heads) {
    PyErr_SetString(PyExc_ValueError, "q must be [T, H_q, D] with H_q a multiple of H_kv");
    goto done;
  }
  if (!operand(a[0], "q", g_bf16, device, 3, shape, 0, &q) || !offsets(a[4], "cu_q", c.seqs, rows, device, &cu)) goto done;
  max_q = cu == NULL || rows < 1 ? 1 : rows;
  if (a[5] != Py_None && !integer(a[5], &max_q)) goto done;
  const double scale = a[6] == Py_None ? pow((double)c.d, -0.5) : PyFloat_AsDouble(a[6]);
  const int causal = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred() || !integer(a[8], &window)) goto done;
  if (a[9] == Py_None) {
    out = empty(a[0], g_bf16, 3, shape, &o.ptr);
    if (out == NULL) goto done;
    o.stride[0] = heads * c.d, o.stride[1] = c.d;
  } else {
    if (!operand(a[9], "out", g_bf16, device, 3, shape, 0, &o)) goto done;
    out = Py_NewRef(a[9]);
  }
  const int64_t lse_shape[2] = {rows, heads};
  if (!optional(a[10], "lse", g_f32, device, 2, lse_shape, &lse)) goto done;
  if (a[11] == Py_None) {
    ws_bytes = (int64_t)prism_kv_attention_workspace_bytes(c.seqs, rows, max_q, c.max_pages, heads, c.heads, c.d, c.block);
    if (ws_bytes > 0 && (held = empty(a[0], g_u8, 1, &ws_bytes, &ws)) == NULL) goto done;
  } else {
    if (!workspace(a[11], device, &ws, &ws_bytes)) goto done;
  }
  if (!optional(a[12], "err", g_i32, device, 1, &kOne, &err) || !stream_of(a[13], device, &stream)) goto done;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_kv_attention(q.ptr, q.stride[0], q.stride[1], c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.table,
                              c.ld_table, c.lens, cu, o.ptr, o.stride[0], o.stride[1], lse, (float)scale, causal, window,
                              c.seqs, rows, max_q, c.num_pages, c.max_pages, heads, c.heads, c.d, c.block, ws,
                              (size_t)ws_bytes, err, stream);
  Py_END_ALLOW_THREADS
  PyObject *none = answer("prism_kv_attention", status);
  done = none != NULL;
  Py_XDECREF(none);
done:
  Py_DECREF(cache);
  Py_XDECREF(held);
  if (!done) Py_CLEAR(out);
  return out;
}

/* w4g_linear(q, a_scale, w4, group_scale, group_offset, residual, out, stream) */
static PyObject *py_w4g(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (!argc_is(nargs, 8)) return NULL;
  int64_t device, group_shape[2];
  Operand q, as, w, s, b = {0}, r = {0}, o;
  void *stream;
  if (!first_operand(a[0], "q", 2, &device, &q) || !shape_of(a[3], "group_scale", 2, group_shape)) return NULL;
  const int64_t m = q.shape[0], k = q.shape[1], n = group_shape[0], groups = group_shape[1];
  if (groups == 0 || k % groups || k % 2) {
    PyErr_SetString(PyExc_ValueError, "q [M, K] and group_scale [N, K/g] do not agree");
    return NULL;
  }
  const int64_t q_shape[2] = {m, k}, w_shape[2] = {n, k / 2}, out_shape[2] = {m, n};
  if (!operand(a[0], "q", g_i8, device, 2, q_shape, 0, &q) || !operand(a[1], "a_scale", g_f32, device, 1, &m, 0, &as) ||
      !operand(a[2], "w4", g_u8, device, 2, w_shape, 0, &w) ||
      !operand(a[3], "group_scale", g_f16, device, 2, group_shape, 0, &s) ||
      (a[4] != Py_None && !operand(a[4], "group_offset", g_f16, device, 2, group_shape, 0, &b)) ||
      (a[5] != Py_None && !operand(a[5], "residual", g_bf16, device, 2, out_shape, 0, &r)) ||
      (a[6] != Py_None && !operand(a[6], "out", g_bf16, device, 2, out_shape, 0, &o)) || !stream_of(a[7], device, &stream))
    return NULL;
  PyObject *out;
  if (a[6] == Py_None) {
    out = empty(a[0], g_bf16, 2, out_shape, &o.ptr);
    if (out == NULL) return NULL;
    o.stride[0] = n;
  } else {
    out = Py_NewRef(a[6]);
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_w4g_linear(q.ptr, q.stride[0], as.ptr, w.ptr, w.stride[0], s.ptr, s.stride[0], b.ptr, b.stride[0], r.ptr,
                            r.stride[0], o.ptr, o.stride[0], m, n, k, k / groups, stream);
  Py_END_ALLOW_THREADS
  PyObject *none = answer("prism_w4g_linear", status);
  if (none == NULL) Py_CLEAR(out);
  Py_XDECREF(none);
  return out;
}

/* token_logprobs(logits, token_ids, top_k, entropy, err, stream) */
static PyObject *py_logprobs(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (!argc_is(nargs, 6)) return NULL;
  int64_t device, ids_shape[2], top_k;
  Operand x, ids;
  void *stream, *err, *lp_ptr, *ent_ptr = NULL, *ti_ptr = NULL, *tl_ptr = NULL;
  PyObject *lp = NULL, *ent = NULL, *ti = NULL, *tl = NULL, *out = NULL;
  if (!first_operand(a[0], "logits", 2, &device, &x) || !shape_of(a[1], "token_ids", 2, ids_shape) ||
      !integer(a[2], &top_k))
    return NULL;
  const int want_entropy = PyObject_IsTrue(a[3]);
  if (want_entropy < 0) return NULL;
  const int64_t rows = x.shape[0], vocab = x.shape[1], n = ids_shape[1];
  const int64_t x_shape[2] = {rows, vocab}, lp_shape[2] = {rows, n}, top_shape[2] = {rows, top_k < 0 ? 0 : top_k};
  ids_shape[0] = rows;
  PyObject *dtype = PyObject_GetAttr(a[0], s_dtype);
  if (dtype == NULL) return NULL;
  const int is_f32 = dtype == g_f32, known = is_f32 || dtype == g_bf16;
  if (!known) PyErr_Format(PyExc_TypeError, "logits must be bfloat16 or float32, got %S", dtype);
  Py_DECREF(dtype);
  if (!known || !operand(a[0], "logits", is_f32 ? g_f32 : g_bf16, device, 2, x_shape, 0, &x) ||
      !operand(a[1], "token_ids", g_i32, device, 2, ids_shape, 0, &ids) ||
      !optional(a[4], "err", g_i32, device, 1, &kOne, &err) || !stream_of(a[5], device, &stream))
    return NULL;
  if ((lp = empty(a[0], g_f32, 2, lp_shape, &lp_ptr)) == NULL) goto done;
  if (want_entropy && (ent = empty(a[0], g_f32, 1, &rows, &ent_ptr)) == NULL) goto done;
  if (top_k != 0 && ((ti = empty(a[0], g_i32, 2, top_shape, &ti_ptr)) == NULL ||
                     (tl = empty(a[0], g_f32, 2, top_shape, &tl_ptr)) == NULL))
    goto done;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_token_logprobs(x.ptr, is_f32, x.stride[0], ids.ptr, ids.stride[0], n, rows, vocab, top_k, lp_ptr, ent_ptr,
                                ti_ptr, tl_ptr, err, stream);
  Py_END_ALLOW_THREADS
  PyObject *none = answer("prism_token_logprobs", status);
  if (none != NULL) {
    Py_DECREF(none);
    out = PyTuple_Pack(4, lp, ent ? ent : Py_None, ti ? ti : Py_None, tl ? tl : Py_None);
  }
done:
  Py_XDECREF(lp);
  Py_XDECREF(ent);
  Py_XDECREF(ti);
  Py_XDECREF(tl);
  return out;
}

/* setup(Tensor, bf16, f16, f32, i8, u8, i32, empty, raw_stream, check) */
static PyObject *py_setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  PyObject **to[10] = {&g_tensor, &g_bf16, &g_f16, &g_f32, &g_i8, &g_u8, &g_i32, &g_empty, &g_raw_stream, &g_check};
  if (!argc_is(n, 10)) return NULL;
  if (!PyType_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "Tensor must be a type");
    return NULL;
  }
  for (int i = 0; i < 10; ++i) Py_XSETREF(*to[i], Py_NewRef(a[i]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, NULL},
    {"w4g_linear", (PyCFunction)(void (*)(void))py_w4g, METH_FASTCALL, NULL},
    {"token_logprobs", (PyCFunction)(void (*)(void))py_logprobs, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__decode(void) {
  struct {
    PyObject **to;
    const char *name;
  } names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},           {&s_device, "device"},
               {&s_stride, "stride"},     {&s_data_ptr, "data_ptr"},     {&s_get_device, "get_device"},
               {&s_cuda_stream, "cuda_stream"}};
  for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
    if ((*names[i].to = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
  if ((s_empty_kw = Py_BuildValue("(ss)", "dtype", "device")) == NULL) return NULL;
  return PyModule_Create(&module);
}

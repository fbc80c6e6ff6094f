// decode_py.cpp -- the Python side of the decode-step entry points, as an
// extension module over libprism.so's C ABI (include/prism.h): reads the
// tensors' addresses, shapes and strides, checks them, allocates outputs and
// workspaces from torch's allocator, and calls.
//
// A decode step is a chain of kernels of 5 to 20 us, so the host time of a call
// is part of its cost.  With the same checks in Python and ctypes a 4-bit linear
// call took 12.8 us, through Python's C API alone 9.4 (torch.empty takes 5 us
// of it after a launch), and here 3.4; token log probabilities 15.2, 14.4, 6.1.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "prism.h"

namespace {

PyObject* g_check = nullptr;   // raises PrismError for a status

constexpr int kMaxRank = 4;

struct Operand {
  void* ptr = nullptr;
  int64_t shape[kMaxRank] = {}, stride[kMaxRank] = {};
};

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    default: return c10::toString(t);
  }
}

const at::Tensor* tensor(PyObject* t, const char* name) {
  if (THPVariable_Check(t)) return &THPVariable_Unpack(t);
  PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return nullptr;
}

int64_t index_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

// The shape, of n dimensions.
bool shape_of(PyObject* obj, const char* name, int n, int64_t* shape) {
  const at::Tensor* t = tensor(obj, name);
  if (t == nullptr) return false;
  if (t->dim() != n) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dims", name, n);
    return false;
  }
  for (int i = 0; i < n; ++i) shape[i] = t->size(i);
  return true;
}

// The CUDA device of the first operand, and its shape of n dimensions.
bool first_operand(PyObject* obj, const char* name, int n, int64_t* device, int64_t* shape) {
  const at::Tensor* t = tensor(obj, name);
  if (t == nullptr) return false;
  *device = index_of(*t);
  if (*device < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be on a CUDA device", name);
    return false;
  }
  return shape_of(obj, name, n, shape);
}

std::string list_of(c10::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// A tensor of this type and shape on this device, its last dimension
// contiguous (dense: all of them).
bool operand(PyObject* obj, const char* name, at::ScalarType type, int64_t device, int n, const int64_t* shape, bool dense,
             Operand* o) {
  const at::Tensor* t = tensor(obj, name);
  if (t == nullptr) return false;
  if (t->scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t->scalar_type()));
    return false;
  }
  if (index_of(*t) != device) {
    PyErr_Format(PyExc_ValueError, "%s must be on cuda:%lld, got %s", name, static_cast<long long>(device),
                 t->device().str().c_str());
    return false;
  }
  const c10::IntArrayRef have = t->sizes();
  if (have != c10::IntArrayRef(shape, n)) {
    PyErr_Format(PyExc_ValueError, "%s must be of shape %s, got %s", name, list_of(c10::IntArrayRef(shape, n)).c_str(),
                 list_of(have).c_str());
    return false;
  }
  if (t->stride(n - 1) != 1 && shape[n - 1] > 1) {
    PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
    return false;
  }
  if (dense && !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return false;
  }
  for (int i = 0; i < n; ++i) o->shape[i] = shape[i], o->stride[i] = t->stride(i);
  o->ptr = t->data_ptr();
  return true;
}

// The address of an optional dense operand, null for None.
bool optional(PyObject* obj, const char* name, at::ScalarType type, int64_t device, int n, const int64_t* shape, void** ptr) {
  Operand o;
  *ptr = nullptr;
  if (obj == Py_None) return true;
  if (!operand(obj, name, type, device, n, shape, true, &o)) return false;
  *ptr = o.ptr;
  return true;
}

// An uninitialised tensor on the device.
at::Tensor empty(at::ScalarType type, int64_t device, int n, const int64_t* shape) {
  return at::Tensor(at::detail::empty_cuda(c10::IntArrayRef(shape, n), type,
                                           c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt));
}

// The stream of a call and the operands' device, torch's current ones for as long
// as `guard` lives: the kernels are launched on that device, and outputs and
// workspaces taken from torch's allocator meanwhile belong to the stream that
// uses them, so that no other stream's work is given their memory.
bool use_stream(PyObject* stream, int64_t device, c10::cuda::OptionalCUDAStreamGuard* guard, void** out) {
  const auto index = static_cast<c10::DeviceIndex>(device);
  if (stream == Py_None) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(index);
    *out = current.stream();
    guard->reset_stream(current);
    return true;
  }
  PyObject* v = PyObject_GetAttrString(stream, "cuda_stream");
  if (v == nullptr) return false;
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (PyErr_Occurred() != nullptr) return false;
  if (PyObject_HasAttrString(stream, "device_index")) {   // torch's streams know theirs; a handle alone is taken as it is
    v = PyObject_GetAttrString(stream, "device_index");
    if (v == nullptr) return false;
    const int64_t of = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred() != nullptr) return false;
    if (of != device) {
      PyErr_Format(PyExc_ValueError, "stream must be of cuda:%lld, got one of cuda:%lld", static_cast<long long>(device),
                   static_cast<long long>(of));
      return false;
    }
  }
  guard->reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(*out), index));
  return true;
}

bool integer(PyObject* v, int64_t* out) {
  *out = PyLong_AsLongLong(v);
  return *out != -1 || PyErr_Occurred() == nullptr;
}

// True for PRISM_OK; else the exception is set.
bool accepted(const char* fn, int status) {
  if (status == PRISM_OK) return true;
  Py_XDECREF(PyObject_CallFunction(g_check, "si", fn, status));
  return false;
}

bool argc_is(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
  return n == want;
}

// A borrowed view of a sequence's items, for as long as this lives.
struct Items {
  PyObject* seq;
  explicit Items(PyObject* obj, const char* what) : seq(PySequence_Fast(obj, what)) {}
  ~Items() { Py_XDECREF(seq); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// The cache's own tensors: its geometry and the addresses of codes, scales,
// page table and lengths.
struct Cache {
  int64_t num_pages, heads, block, d, seqs, max_pages, ld_table;
  void *k_codes, *v_codes, *k_scale, *v_scale, *table, *lens;
};

bool read_cache(const Items& t, PyObject* page_table, PyObject* seq_lens, int64_t device, Cache* c) {
  if (t.size() < 4) {
    PyErr_SetString(PyExc_ValueError, "cache must have k_codes, v_codes, k_scale, v_scale");
    return false;
  }
  int64_t shape[4], table_shape[2];
  Operand kc, vc, ks, vs, table, lens;
  if (!shape_of(t[0], "k_codes", 4, shape) || !shape_of(page_table, "page_table", 2, table_shape) ||
      !operand(t[0], "k_codes", at::kChar, device, 4, shape, true, &kc) ||
      !operand(t[1], "v_codes", at::kChar, device, 4, shape, true, &vc) ||
      !operand(t[2], "k_scale", at::kFloat, device, 2, shape, true, &ks) ||
      !operand(t[3], "v_scale", at::kFloat, device, 2, shape, true, &vs) ||
      !operand(page_table, "page_table", at::kInt, device, 2, table_shape, false, &table) ||
      !operand(seq_lens, "seq_lens", at::kInt, device, 1, table_shape, false, &lens))
    return false;
  *c = Cache{shape[0], shape[1], shape[2],  shape[3], table_shape[0], table_shape[1], table.stride[0],
             kc.ptr,   vc.ptr,   ks.ptr,    vs.ptr,   table.ptr,      lens.ptr};
  return true;
}

bool offsets(PyObject* cu, const char* name, int64_t seqs, int64_t rows, int64_t device, void** ptr) {
  const int64_t n = seqs + 1;
  Operand o;
  *ptr = nullptr;
  if (cu == Py_None) {
    if (rows != seqs) PyErr_Format(PyExc_ValueError, "without %s there is one row for each sequence", name);
    return rows == seqs;
  }
  if (!operand(cu, name, at::kInt, device, 1, &n, false, &o)) return false;
  *ptr = o.ptr;
  return true;
}

constexpr int64_t kOne = 1;

// append(k, v, cache, page_table, seq_lens, cu_new, max_new, err, stream)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc_is(n, 9)) return nullptr;
  int64_t device, first[3], max_new;
  Operand k, v, ko, vo;
  Cache c;
  void *cu, *err, *stream;
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (!first_operand(a[0], "k", 3, &device, first)) return nullptr;
  const Items cache(a[2], "cache must be a sequence of tensors");
  if (cache.seq == nullptr || !read_cache(cache, a[3], a[4], device, &c)) return nullptr;
  if (cache.size() < 6) {
    PyErr_SetString(PyExc_ValueError, "cache must have k_open and v_open");
    return nullptr;
  }
  const int64_t rows = first[0], shape[3] = {rows, c.heads, c.d}, open[4] = {c.seqs, c.heads, c.block, c.d};
  if (!operand(a[0], "k", at::kBFloat16, device, 3, shape, false, &k) ||
      !operand(a[1], "v", at::kBFloat16, device, 3, shape, false, &v) ||
      !operand(cache[4], "k_open", at::kBFloat16, device, 4, open, true, &ko) ||
      !operand(cache[5], "v_open", at::kBFloat16, device, 4, open, true, &vo) ||
      !offsets(a[5], "cu_new", c.seqs, rows, device, &cu))
    return nullptr;
  max_new = cu == nullptr || rows < 1 ? 1 : rows;
  if (a[6] != Py_None && !integer(a[6], &max_new)) return nullptr;
  if (!optional(a[7], "err", at::kInt, device, 1, &kOne, &err) || !use_stream(a[8], device, &guard, &stream)) return nullptr;
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_kv_append(k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1],
                           static_cast<int8_t*>(c.k_codes), static_cast<int8_t*>(c.v_codes), static_cast<float*>(c.k_scale),
                           static_cast<float*>(c.v_scale), ko.ptr, vo.ptr, static_cast<int32_t*>(c.table), c.ld_table,
                           static_cast<int32_t*>(c.lens), static_cast<int32_t*>(cu), c.seqs, rows, max_new, c.num_pages,
                           c.max_pages, c.heads, c.d, c.block, static_cast<int32_t*>(err), stream);
  Py_END_ALLOW_THREADS
  if (!accepted("prism_kv_append", status)) return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// attention(q, cache, page_table, seq_lens, cu_q, max_q, scale, causal, window, out, lse, workspace, err, stream)
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc_is(n, 14)) return nullptr;
  int64_t device, first[3], max_q, window, ws_bytes = 0;
  Operand q, o;
  Cache c;
  void *cu, *lse, *err, *stream, *ws = nullptr;
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (!first_operand(a[0], "q", 3, &device, first)) return nullptr;
  const Items cache(a[1], "cache must be a sequence of tensors");
  if (cache.seq == nullptr || !read_cache(cache, a[2], a[3], device, &c)) return nullptr;
  const int64_t rows = first[0], heads = first[1], shape[3] = {rows, heads, c.d}, lse_shape[2] = {rows, heads};
  if (first[2] != c.d || heads == 0 || c.heads == 0 || heads % c.heads) {
    PyErr_SetString(PyExc_ValueError, "q must be [T, H_q, D] with H_q a multiple of H_kv");
    return nullptr;
  }
  if (!operand(a[0], "q", at::kBFloat16, device, 3, shape, false, &q) ||
      !offsets(a[4], "cu_q", c.seqs, rows, device, &cu))
    return nullptr;
  max_q = cu == nullptr || rows < 1 ? 1 : rows;
  if (a[5] != Py_None && !integer(a[5], &max_q)) return nullptr;
  const double scale = a[6] == Py_None ? std::pow(static_cast<double>(c.d), -0.5) : PyFloat_AsDouble(a[6]);
  const int causal = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred() != nullptr || !integer(a[8], &window)) return nullptr;
  if (a[9] != Py_None && !operand(a[9], "out", at::kBFloat16, device, 3, shape, false, &o)) return nullptr;
  if (!optional(a[10], "lse", at::kFloat, device, 2, lse_shape, &lse)) return nullptr;
  if (!optional(a[12], "err", at::kInt, device, 1, &kOne, &err) || !use_stream(a[13], device, &guard, &stream)) return nullptr;
  at::Tensor held, made;
  if (a[11] != Py_None) {
    const at::Tensor* w = tensor(a[11], "workspace");
    if (w == nullptr) return nullptr;
    if (index_of(*w) != device || !w->is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:%lld", static_cast<long long>(device));
      return nullptr;
    }
    ws = w->data_ptr();
    ws_bytes = static_cast<int64_t>(w->nbytes());
  } else {
    ws_bytes = static_cast<int64_t>(
        prism_kv_attention_workspace_bytes(c.seqs, rows, max_q, c.max_pages, heads, c.heads, c.d, c.block));
    if (ws_bytes > 0) {
      held = empty(at::kByte, device, 1, &ws_bytes);
      ws = held.data_ptr();
    }
  }
  if (a[9] == Py_None) {
    made = empty(at::kBFloat16, device, 3, shape);
    o.ptr = made.data_ptr();
    o.stride[0] = heads * c.d, o.stride[1] = c.d;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_kv_attention(q.ptr, q.stride[0], q.stride[1], static_cast<int8_t*>(c.k_codes),
                              static_cast<int8_t*>(c.v_codes), static_cast<float*>(c.k_scale),
                              static_cast<float*>(c.v_scale), static_cast<int32_t*>(c.table), c.ld_table,
                              static_cast<int32_t*>(c.lens), static_cast<int32_t*>(cu), o.ptr, o.stride[0], o.stride[1],
                              static_cast<float*>(lse), static_cast<float>(scale), causal, window, c.seqs, rows, max_q,
                              c.num_pages, c.max_pages, heads, c.heads, c.d, c.block, ws, static_cast<size_t>(ws_bytes),
                              static_cast<int32_t*>(err), stream);
  Py_END_ALLOW_THREADS
  if (!accepted("prism_kv_attention", status)) return nullptr;
  return a[9] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[9]);
  END_HANDLE_TH_ERRORS
}

// w4g_linear(q, a_scale, w4, group_scale, group_offset, residual, out, stream)
PyObject* py_w4g(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!argc_is(nargs, 8)) return nullptr;
  int64_t device, first[2], group_shape[2];
  Operand q, as, w, s, b, r, o;
  void* stream;
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (!first_operand(a[0], "q", 2, &device, first) || !shape_of(a[3], "group_scale", 2, group_shape)) return nullptr;
  const int64_t m = first[0], k = first[1], n = group_shape[0], groups = group_shape[1];
  if (groups == 0 || k % groups || k % 2) {
    PyErr_SetString(PyExc_ValueError, "q [M, K] and group_scale [N, K/g] do not agree");
    return nullptr;
  }
  const int64_t w_shape[2] = {n, k / 2}, out_shape[2] = {m, n};
  if (!operand(a[0], "q", at::kChar, device, 2, first, false, &q) ||
      !operand(a[1], "a_scale", at::kFloat, device, 1, &m, false, &as) ||
      !operand(a[2], "w4", at::kByte, device, 2, w_shape, false, &w) ||
      !operand(a[3], "group_scale", at::kHalf, device, 2, group_shape, false, &s) ||
      (a[4] != Py_None && !operand(a[4], "group_offset", at::kHalf, device, 2, group_shape, false, &b)) ||
      (a[5] != Py_None && !operand(a[5], "residual", at::kBFloat16, device, 2, out_shape, false, &r)) ||
      (a[6] != Py_None && !operand(a[6], "out", at::kBFloat16, device, 2, out_shape, false, &o)) ||
      !use_stream(a[7], device, &guard, &stream))
    return nullptr;
  at::Tensor made;
  if (a[6] == Py_None) {
    made = empty(at::kBFloat16, device, 2, out_shape);
    o.ptr = made.data_ptr();
    o.stride[0] = n;
  }
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_w4g_linear(static_cast<int8_t*>(q.ptr), q.stride[0], static_cast<float*>(as.ptr),
                            static_cast<uint8_t*>(w.ptr), w.stride[0], static_cast<uint16_t*>(s.ptr), s.stride[0],
                            static_cast<uint16_t*>(b.ptr), b.stride[0], r.ptr,
                            r.stride[0], o.ptr, o.stride[0], m, n, k, k / groups, stream);
  Py_END_ALLOW_THREADS
  if (!accepted("prism_w4g_linear", status)) return nullptr;
  return a[6] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[6]);
  END_HANDLE_TH_ERRORS
}

// token_logprobs(logits, token_ids, top_k, entropy, err, stream)
PyObject* py_logprobs(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (!argc_is(nargs, 6)) return nullptr;
  int64_t device, first[2], ids_shape[2], top_k;
  Operand x, ids;
  void *stream, *err;
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (!first_operand(a[0], "logits", 2, &device, first) || !shape_of(a[1], "token_ids", 2, ids_shape) ||
      !integer(a[2], &top_k))
    return nullptr;
  const int want_entropy = PyObject_IsTrue(a[3]);
  if (want_entropy < 0) return nullptr;
  const int64_t rows = first[0], vocab = first[1], n = ids_shape[1];
  const int64_t lp_shape[2] = {rows, n}, top_shape[2] = {rows, top_k < 0 ? 0 : top_k};
  ids_shape[0] = rows;
  const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) {
    PyErr_Format(PyExc_TypeError, "logits must be bfloat16 or float32, got %s", type_name(type));
    return nullptr;
  }
  if (!operand(a[0], "logits", type, device, 2, first, false, &x) ||
      !operand(a[1], "token_ids", at::kInt, device, 2, ids_shape, false, &ids) ||
      !optional(a[4], "err", at::kInt, device, 1, &kOne, &err) || !use_stream(a[5], device, &guard, &stream))
    return nullptr;
  at::Tensor lp = empty(at::kFloat, device, 2, lp_shape), ent, ti, tl;
  if (want_entropy) ent = empty(at::kFloat, device, 1, &rows);
  if (top_k != 0) ti = empty(at::kInt, device, 2, top_shape), tl = empty(at::kFloat, device, 2, top_shape);
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = prism_token_logprobs(x.ptr, type == at::kFloat, x.stride[0], static_cast<int32_t*>(ids.ptr), ids.stride[0], n,
                                rows, vocab, top_k, static_cast<float*>(ptr(lp)), static_cast<float*>(ptr(ent)),
                                static_cast<int32_t*>(ptr(ti)), static_cast<float*>(ptr(tl)), static_cast<int32_t*>(err),
                                stream);
  Py_END_ALLOW_THREADS
  if (!accepted("prism_token_logprobs", status)) return nullptr;
  at::Tensor* const outs[4] = {&lp, &ent, &ti, &tl};
  PyObject* tuple = PyTuple_New(4);
  for (int i = 0; tuple != nullptr && i < 4; ++i) {
    PyObject* v = outs[i]->defined() ? THPVariable_Wrap(std::move(*outs[i])) : Py_NewRef(Py_None);
    if (v == nullptr) Py_CLEAR(tuple);
    else PyTuple_SET_ITEM(tuple, i, v);
  }
  return tuple;
  END_HANDLE_TH_ERRORS
}

// setup(check): check(name, status) raises for a status
PyObject* py_setup(PyObject*, PyObject* check) {
  Py_XSETREF(g_check, Py_NewRef(check));
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"setup", py_setup, METH_O, nullptr},
                         {"append", fast(py_append), METH_FASTCALL, nullptr},
                         {"attention", fast(py_attention), METH_FASTCALL, nullptr},
                         {"w4g_linear", fast(py_w4g), METH_FASTCALL, nullptr},
                         {"token_logprobs", fast(py_logprobs), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&module); }

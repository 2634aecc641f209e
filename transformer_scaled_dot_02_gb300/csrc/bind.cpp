// The paged helpers' argument handling as a CPython extension: checks the
// tensors of one call and passes their addresses to the C entry points, whose
// addresses Python hands over once (bind).
//
// A step for a few sequences takes the GPU 3 to 8 us, and checking eight
// tensors attribute by attribute in Python and converting 24 arguments
// through ctypes takes about as long: 6 and 2.4 us of the 10 us that an append
// of 8 tokens took from Python.  The checks are the ones that the C entry
// points cannot make themselves: types, shapes, layout, device.
//
// Every function returns its output, or the library's status as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <new>

#include "sdpa.h"

namespace {

decltype(&sdpa_paged_append) append_entry = nullptr;
decltype(&sdpa_paged_forward) forward_entry = nullptr;
decltype(&sdpa_paged_workspace_size) workspace_entry = nullptr;
decltype(&sdpa_paged4_append) append4_entry = nullptr;
decltype(&sdpa_paged4_read) read4_entry = nullptr;
decltype(&sdpa_paged4_forward) forward4_entry = nullptr;
decltype(&sdpa_paged4_workspace_size) workspace4_entry = nullptr;

constexpr int kInvalid = SDPA_ERR_INVALID_ARG;

const at::Tensor* tensor_of(PyObject* x) {
  if (!THPVariable_Check(x)) {
    PyErr_Format(PyExc_TypeError, "expected a torch tensor, got %s", Py_TYPE(x)->tp_name);
    return nullptr;
  }
  return &THPVariable_Unpack(x);
}

// A dense strided tensor of this type on this CUDA device.
bool plain(const at::Tensor& x, at::ScalarType type, int device) {
  return x.layout() == at::kStrided && x.is_cuda() && x.get_device() == device && x.scalar_type() == type;
}

struct Cache {
  int device, b, h_kv, d, page, n_pages, per_seq;
  const void *table, *starts, *lengths;
  void *k, *v;
};

// The pages, table and lengths of a call (on the current device).  d4: columns of
// a row of a cache in 4 bits, 0 for one in bf16.
bool check_cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& starts,
                 const at::Tensor& lengths, int64_t d4, Cache* c) {
  if (!k.is_cuda()) return false;
  c->device = static_cast<int>(k.get_device());
  if (c->device != c10::cuda::current_device()) return false;
  const at::ScalarType held = d4 > 0 ? at::kByte : at::kBFloat16;
  if (!plain(k, held, c->device) || !plain(v, held, c->device) || !plain(table, at::kInt, c->device) ||
      !plain(starts, at::kInt, c->device) || !plain(lengths, at::kInt, c->device))
    return false;
  if (k.dim() != 4 || v.sizes() != k.sizes() || table.dim() != 2 || starts.dim() != 1 || lengths.dim() != 1)
    return false;
  const int64_t b = table.size(0);
  if (starts.size(0) != b + 1 || lengths.size(0) != b) return false;
  if (!k.is_contiguous() || !v.is_contiguous() || !table.is_contiguous() || !starts.is_contiguous() ||
      !lengths.is_contiguous())
    return false;
  for (const int64_t n : k.sizes())
    if (n > INT32_MAX) return false;
  if (b > INT32_MAX || table.size(1) > INT32_MAX) return false;
  c->b = static_cast<int>(b);
  c->per_seq = static_cast<int>(table.size(1));
  c->n_pages = static_cast<int>(k.size(0));
  c->h_kv = static_cast<int>(k.size(1));
  c->page = static_cast<int>(k.size(2));
  if (d4 > 0 && (d4 > INT32_MAX / 16 || d4 % 16 != 0 || 16 * k.size(3) != 9 * d4)) return false;
  c->d = static_cast<int>(d4 > 0 ? d4 : k.size(3));
  c->table = table.const_data_ptr();
  c->starts = starts.const_data_ptr();
  c->lengths = lengths.const_data_ptr();
  c->k = k.data_ptr();
  c->v = v.data_ptr();
  return true;
}

// Do the keys' and the values' pages share memory?  The attention may read them so,
// the append would store both to one place.
bool pages_overlap(const at::Tensor& k, const at::Tensor& v) {
  const auto a = reinterpret_cast<uintptr_t>(k.const_data_ptr()), b = reinterpret_cast<uintptr_t>(v.const_data_ptr());
  return a < b + v.nbytes() && b < a + k.nbytes();
}

// Packed rows [n_tokens, heads, d] whose heads are dense; the stride from token
// to token (a single token's says nothing, and no stride of a tensor without elements does).
bool check_rows(const at::Tensor& x, int64_t n_tokens, int64_t heads, const Cache& c, long long* stride) {
  if (!plain(x, at::kBFloat16, c.device) || x.dim() != 3 || x.size(0) != n_tokens || x.size(1) != heads ||
      x.size(2) != c.d || (x.numel() > 0 && (x.stride(2) != 1 || (x.stride(1) != c.d && heads != 1))))
    return false;
  *stride = n_tokens > 1 ? x.stride(0) : heads * c.d;
  return true;
}

// Runs f, turning C++ exceptions (torch's own errors) into Python's.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// A Python int that fits 32 bits.
bool int_of(PyObject* x, int* value) {
  const long v = PyLong_AsLong(x);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "expected an int of 32 bits");
    return false;
  }
  *value = static_cast<int>(v);
  return true;
}

PyObject* status_object(int status) { return PyLong_FromLong(status); }

PyObject* returned(PyObject* given, const at::Tensor& made) {
  if (given == Py_None && made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

bool counted(const char* name, Py_ssize_t n, Py_ssize_t want, bool bound) {
  if (!bound) PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
  else if (n != want) PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
  return bound && n == want;
}

// append(q, k, v, k_pages, v_pages, page_table, q_starts, kv_lengths, rope_freqs, interleaved, q_out),
// append4(..., interleaved, k_exp, v_exp, q_out)
template <bool k4>
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kOut = k4 ? 12 : 10;
  if (!counted(k4 ? "append4" : "append", n, kOut + 1, k4 ? append4_entry != nullptr : append_entry != nullptr))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x[8];
    for (int i = 1; i < 8; ++i)
      if ((x[i] = tensor_of(a[i])) == nullptr) return nullptr;
    const at::Tensor &k = *x[1], &v = *x[2];
    Cache c;
    int k_exp = 0, v_exp = 0;
    if (k4 && (!int_of(a[10], &k_exp) || !int_of(a[11], &v_exp))) return nullptr;
    if (k.dim() != 3 || (k4 && k.size(2) < 1) ||
        !check_cache(*x[3], *x[4], *x[5], *x[6], *x[7], k4 ? k.size(2) : 0, &c) || pages_overlap(*x[3], *x[4]))
      return status_object(kInvalid);
    const int64_t t = k.size(0);
    long long q_stride = 0, k_stride, v_stride, out_stride;
    if (t > INT32_MAX || !check_rows(k, t, c.h_kv, c, &k_stride) || !check_rows(v, t, c.h_kv, c, &v_stride))
      return status_object(kInvalid);
    int64_t h = c.h_kv;
    const void* q_ptr = nullptr;
    void* out_ptr = nullptr;
    at::Tensor made;
    if (a[0] != Py_None) {
      const at::Tensor* q = tensor_of(a[0]);
      if (q == nullptr) return nullptr;
      if (q->dim() != 3) return status_object(kInvalid);
      h = q->size(1);
      if (h > INT32_MAX || !check_rows(*q, t, h, c, &q_stride)) return status_object(kInvalid);
      q_ptr = q->const_data_ptr();
      if (a[kOut] == Py_None) {
        made = at::empty({t, h, c.d}, k.options());
        out_ptr = made.data_ptr();
      } else {
        const at::Tensor* out = tensor_of(a[kOut]);
        if (out == nullptr) return nullptr;
        if (!check_rows(*out, t, h, c, &out_stride) || !out->is_contiguous()) return status_object(kInvalid);
        out_ptr = out->data_ptr();
      }
    } else if (a[kOut] != Py_None) {
      return status_object(kInvalid);
    }
    const float* freqs = nullptr;
    int d_rot = 0;
    if (a[8] != Py_None) {
      const at::Tensor* f = tensor_of(a[8]);
      if (f == nullptr) return nullptr;
      if (!plain(*f, at::kFloat, c.device) || !f->is_contiguous() || f->numel() > c.d) return status_object(kInvalid);
      freqs = static_cast<const float*>(f->const_data_ptr());
      d_rot = static_cast<int>(2 * f->numel());
    }
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) return nullptr;
    const void *k_ptr = k.const_data_ptr(), *v_ptr = v.const_data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    if constexpr (k4)
      status = append4_entry(q_ptr, k_ptr, v_ptr, out_ptr, c.k, c.v, c.b, static_cast<int>(t), static_cast<int>(h),
                             c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                             static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                             k_stride, v_stride, freqs, d_rot, interleaved, k_exp, v_exp, stream);
    else
      status = append_entry(q_ptr, k_ptr, v_ptr, out_ptr, c.k, c.v, c.b, static_cast<int>(t), static_cast<int>(h),
                            c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                            static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                            k_stride, v_stride, freqs, d_rot, interleaved, stream);
    Py_END_ALLOW_THREADS
    return status != 0 ? status_object(status) : returned(a[kOut], made);
  });
}

// forward(q, k_pages, v_pages, page_table, q_starts, kv_lengths, scale, out, workspace),
// forward4(..., scale, k_exp, v_exp, window, sinks, out, workspace);
// a workspace that is not given is allocated once the tensors have been checked
template <bool k4>
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kOut = k4 ? 11 : 7, kWorkspace = kOut + 1;
  if (!counted(k4 ? "forward4" : "forward", n, kWorkspace + 1, k4 ? forward4_entry != nullptr : forward_entry != nullptr))
    return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x[6];
    for (int i = 0; i < 6; ++i)
      if ((x[i] = tensor_of(a[i])) == nullptr) return nullptr;
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const at::Tensor& q = *x[0];
    Cache c;
    int k_exp = 0, v_exp = 0, window = 0, sinks = 0;
    if (k4 && (!int_of(a[7], &k_exp) || !int_of(a[8], &v_exp) || !int_of(a[9], &window) || !int_of(a[10], &sinks)))
      return nullptr;
    if (q.dim() != 3 || (k4 && q.size(2) < 1) ||
        !check_cache(*x[1], *x[2], *x[3], *x[4], *x[5], k4 ? q.size(2) : 0, &c))
      return status_object(kInvalid);
    const int64_t t = q.size(0), h = q.size(1);
    long long q_stride, out_stride;
    if (t > INT32_MAX || h > INT32_MAX || !check_rows(q, t, h, c, &q_stride)) return status_object(kInvalid);
    at::Tensor made, made_ws;
    void *out_ptr, *ws = nullptr;
    if (a[kOut] == Py_None) {
      made = at::empty({t, h, c.d}, q.options());
      out_ptr = made.data_ptr();
    } else {
      const at::Tensor* out = tensor_of(a[kOut]);
      if (out == nullptr) return nullptr;
      if (!check_rows(*out, t, h, c, &out_stride) || !out->is_contiguous()) return status_object(kInvalid);
      out_ptr = out->data_ptr();
    }
    size_t ws_bytes = 0;
    if (a[kWorkspace] != Py_None) {
      const at::Tensor* w = tensor_of(a[kWorkspace]);
      if (w == nullptr) return nullptr;
      if (!plain(*w, w->scalar_type(), c.device) || !w->is_contiguous()) return status_object(kInvalid);
      ws = w->data_ptr();
      ws_bytes = w->nbytes();
    } else {
      ws_bytes = (k4 ? workspace4_entry : workspace_entry)(c.b, static_cast<int>(t), static_cast<int>(h), c.h_kv, c.d,
                                                          c.page, c.per_seq);
      if (ws_bytes > 0) {
        made_ws = at::empty({static_cast<int64_t>(ws_bytes)}, q.options().dtype(at::kByte));
        ws = made_ws.data_ptr();
      }
    }
    const void* q_ptr = q.const_data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    if constexpr (k4)
      status = forward4_entry(q_ptr, c.k, c.v, out_ptr, ws, ws_bytes, c.b, static_cast<int>(t), static_cast<int>(h),
                              c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                              static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                              static_cast<float>(scale), k_exp, v_exp, window, sinks, stream);
    else
      status = forward_entry(q_ptr, c.k, c.v, out_ptr, ws, ws_bytes, c.b, static_cast<int>(t), static_cast<int>(h),
                             c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                             static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                             static_cast<float>(scale), stream);
    Py_END_ALLOW_THREADS
    return status != 0 ? status_object(status) : returned(a[kOut], made);
  });
}

// read4(k_pages, v_pages, page_table, q_starts, kv_lengths, k_out, v_out, k_exp, v_exp)
PyObject* read4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted("read4", n, 9, read4_entry != nullptr)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x[7];
    for (int i = 0; i < 7; ++i)
      if ((x[i] = tensor_of(a[i])) == nullptr) return nullptr;
    int k_exp, v_exp;
    if (!int_of(a[7], &k_exp) || !int_of(a[8], &v_exp)) return nullptr;
    const at::Tensor &k = *x[5], &v = *x[6];
    Cache c;
    if (k.dim() != 3 || k.size(2) < 1 || !check_cache(*x[0], *x[1], *x[2], *x[3], *x[4], k.size(2), &c))
      return status_object(kInvalid);
    const int64_t t = k.size(0);
    long long stride;
    if (t > INT32_MAX || !check_rows(k, t, c.h_kv, c, &stride) || !check_rows(v, t, c.h_kv, c, &stride) ||
        !k.is_contiguous() || !v.is_contiguous())
      return status_object(kInvalid);
    void *k_ptr = k.data_ptr(), *v_ptr = v.data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = read4_entry(c.k, c.v, k_ptr, v_ptr, c.b, static_cast<int>(t), c.h_kv, c.d, c.page, c.n_pages, c.per_seq,
                         static_cast<const int32_t*>(c.table), static_cast<const int32_t*>(c.starts),
                         static_cast<const int32_t*>(c.lengths), k_exp, v_exp, stream);
    Py_END_ALLOW_THREADS
    return status_object(status);
  });
}

// bind(append, forward, workspace, append4, read4, forward4, workspace4): the
// addresses of sdpa_paged_append, sdpa_paged_forward, sdpa_paged_workspace_size and
// of those of the cache in 4 bits
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted("bind", n, 7, true)) return nullptr;
  void* x[7];
  for (int i = 0; i < 7; ++i) x[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  append_entry = reinterpret_cast<decltype(append_entry)>(x[0]);
  forward_entry = reinterpret_cast<decltype(forward_entry)>(x[1]);
  workspace_entry = reinterpret_cast<decltype(workspace_entry)>(x[2]);
  append4_entry = reinterpret_cast<decltype(append4_entry)>(x[3]);
  read4_entry = reinterpret_cast<decltype(read4_entry)>(x[4]);
  forward4_entry = reinterpret_cast<decltype(forward4_entry)>(x[5]);
  workspace4_entry = reinterpret_cast<decltype(workspace4_entry)>(x[6]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(f); }

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"append", fast(append<false>), METH_FASTCALL, nullptr},
    {"append4", fast(append<true>), METH_FASTCALL, nullptr},
    {"read4", fast(read4), METH_FASTCALL, nullptr},
    {"forward", fast(forward<false>), METH_FASTCALL, nullptr},
    {"forward4", fast(forward<true>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Argument handling of the paged helpers.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
  PyObject* m = PyModule_Create(&module);
  // the torch that this was compiled against: Python compares it with its own
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", SDPA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}

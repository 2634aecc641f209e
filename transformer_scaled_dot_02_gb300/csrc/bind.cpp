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

// The pages, table and lengths of a call (on the current device).
bool check_cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& starts,
                 const at::Tensor& lengths, Cache* c) {
  if (!k.is_cuda()) return false;
  c->device = static_cast<int>(k.get_device());
  if (c->device != c10::cuda::current_device()) return false;
  if (!plain(k, at::kBFloat16, c->device) || !plain(v, at::kBFloat16, c->device) ||
      !plain(table, at::kInt, c->device) || !plain(starts, at::kInt, c->device) ||
      !plain(lengths, at::kInt, c->device))
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
  c->d = static_cast<int>(k.size(3));
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
// to token (a single token's says nothing).
bool check_rows(const at::Tensor& x, int64_t n_tokens, int64_t heads, const Cache& c, long long* stride) {
  if (!plain(x, at::kBFloat16, c.device) || x.dim() != 3 || x.size(0) != n_tokens || x.size(1) != heads ||
      x.size(2) != c.d || x.stride(2) != 1 || (x.stride(1) != c.d && heads != 1))
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

// append(q, k, v, k_pages, v_pages, page_table, q_starts, kv_lengths, rope_freqs, interleaved, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted("append", n, 11, append_entry != nullptr)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x[8];
    for (int i = 1; i < 8; ++i)
      if ((x[i] = tensor_of(a[i])) == nullptr) return nullptr;
    const at::Tensor &k = *x[1], &v = *x[2];
    Cache c;
    if (!check_cache(*x[3], *x[4], *x[5], *x[6], *x[7], &c) || k.dim() != 3 || pages_overlap(*x[3], *x[4]))
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
      if (a[10] == Py_None) {
        made = at::empty({t, h, c.d}, k.options());
        out_ptr = made.data_ptr();
      } else {
        const at::Tensor* out = tensor_of(a[10]);
        if (out == nullptr) return nullptr;
        if (!check_rows(*out, t, h, c, &out_stride) || !out->is_contiguous()) return status_object(kInvalid);
        out_ptr = out->data_ptr();
      }
    } else if (a[10] != Py_None) {
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
    status = append_entry(q_ptr, k_ptr, v_ptr, out_ptr, c.k, c.v, c.b, static_cast<int>(t), static_cast<int>(h),
                          c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                          static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                          k_stride, v_stride, freqs, d_rot, interleaved, stream);
    Py_END_ALLOW_THREADS
    return status != 0 ? status_object(status) : returned(a[10], made);
  });
}

// forward(q, k_pages, v_pages, page_table, q_starts, kv_lengths, scale, out, workspace);
// a workspace that is not given is allocated once the tensors have been checked
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted("forward", n, 9, forward_entry != nullptr)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* x[6];
    for (int i = 0; i < 6; ++i)
      if ((x[i] = tensor_of(a[i])) == nullptr) return nullptr;
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const at::Tensor& q = *x[0];
    Cache c;
    if (!check_cache(*x[1], *x[2], *x[3], *x[4], *x[5], &c) || q.dim() != 3) return status_object(kInvalid);
    const int64_t t = q.size(0), h = q.size(1);
    long long q_stride, out_stride;
    if (t > INT32_MAX || h > INT32_MAX || !check_rows(q, t, h, c, &q_stride)) return status_object(kInvalid);
    at::Tensor made, made_ws;
    void *out_ptr, *ws = nullptr;
    if (a[7] == Py_None) {
      made = at::empty({t, h, c.d}, q.options());
      out_ptr = made.data_ptr();
    } else {
      const at::Tensor* out = tensor_of(a[7]);
      if (out == nullptr) return nullptr;
      if (!check_rows(*out, t, h, c, &out_stride) || !out->is_contiguous()) return status_object(kInvalid);
      out_ptr = out->data_ptr();
    }
    size_t ws_bytes = 0;
    if (a[8] != Py_None) {
      const at::Tensor* w = tensor_of(a[8]);
      if (w == nullptr) return nullptr;
      if (!plain(*w, w->scalar_type(), c.device) || !w->is_contiguous()) return status_object(kInvalid);
      ws = w->data_ptr();
      ws_bytes = w->nbytes();
    } else {
      ws_bytes = workspace_entry(c.b, static_cast<int>(t), static_cast<int>(h), c.h_kv, c.d, c.page, c.per_seq);
      if (ws_bytes > 0) {
        made_ws = at::empty({static_cast<int64_t>(ws_bytes)}, q.options().dtype(at::kByte));
        ws = made_ws.data_ptr();
      }
    }
    const void* q_ptr = q.const_data_ptr();
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = forward_entry(q_ptr, c.k, c.v, out_ptr, ws, ws_bytes, c.b, static_cast<int>(t), static_cast<int>(h),
                           c.h_kv, c.d, c.page, c.n_pages, c.per_seq, static_cast<const int32_t*>(c.table),
                           static_cast<const int32_t*>(c.starts), static_cast<const int32_t*>(c.lengths), q_stride,
                           static_cast<float>(scale), stream);
    Py_END_ALLOW_THREADS
    return status != 0 ? status_object(status) : returned(a[7], made);
  });
}

// bind(append, forward, workspace): the addresses of sdpa_paged_append,
// sdpa_paged_forward and sdpa_paged_workspace_size
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted("bind", n, 3, true)) return nullptr;
  void *x = PyLong_AsVoidPtr(a[0]), *y = PyLong_AsVoidPtr(a[1]), *z = PyLong_AsVoidPtr(a[2]);
  if (PyErr_Occurred()) return nullptr;
  append_entry = reinterpret_cast<decltype(append_entry)>(x);
  forward_entry = reinterpret_cast<decltype(forward_entry)>(y);
  workspace_entry = reinterpret_cast<decltype(workspace_entry)>(z);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(append), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(forward), METH_FASTCALL, nullptr},
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

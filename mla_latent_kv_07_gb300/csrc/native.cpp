// native.cpp -- the host path of the paged calls that a serving loop makes for every
// layer of every step, as a Python extension: checks of the tensors, outputs from
// the caching allocator and the call into libmla, without Python in between.
//
// Each function takes what its binding was given and answers with the outputs
// (a tuple), with a library status that is not MLA_OK (an int), or with None
// where something is not the plain case: a tensor of another type, shape, layout
// or device, a pool on another device than the current one, a given stream.  The
// binding then goes through the call itself, in Python, and says what is wrong or
// does what is asked.  Measured on the host of a GB300: paged_append_rotary of one
// token 17.6 us in Python, 5.6 here (3.8 of them the launch).
//
// Library entry points are bound by address, so the extension and the ctypes
// binding share one loaded libmla.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mla.h"

namespace {

struct Library {
  decltype(&mla_paged_append_rotary) append_rotary = nullptr;
  decltype(&mla_paged_read) read = nullptr;
  decltype(&mla_paged_decode_window) decode_window = nullptr;
  decltype(&mla_paged_window_workspace_size) window_workspace_size = nullptr;
} lib;

// ------------------------------------------------------------- arguments
// Every getter clears `ok` where the argument is not the plain case.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  bool ok = true;
  int dev = -1;

  PyObject* next() {
    if (i >= n) {
      ok = false;
      return Py_None;
    }
    return a[i++];
  }
  bool none() { return i < n && a[i] == Py_None ? (++i, true) : false; }
  const at::Tensor* tensor(at::ScalarType type) {
    PyObject* o = next();
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  // its columns side by side; the other dimensions anywhere
  const at::Tensor* rows(at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(type);
    if (t && (t->sizes() != shape || t->strides().back() != 1)) ok = false;
    return t;
  }
  const at::Tensor* dense(at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(type);
    if (t && (t->sizes() != shape || !t->is_contiguous())) ok = false;
    return t;
  }
  // a given output, or a new one
  at::Tensor output(at::ScalarType type, at::IntArrayRef shape) {
    if (!none()) {
      const at::Tensor* t = dense(type, shape);
      return ok ? *t : at::Tensor();
    }
    return ok ? make(type, shape) : at::Tensor();
  }
  at::Tensor make(at::ScalarType type, at::IntArrayRef shape) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
  }
  long long integer(long long lo, long long hi) {
    PyObject* o = next();
    int over = 0;
    const long long v = PyLong_Check(o) ? PyLong_AsLongLongAndOverflow(o, &over) : (ok = false, 0);
    if (over || v < lo || v > hi) ok = false;
    return v;
  }
  int32_t int32() { return (int32_t)integer(INT32_MIN, INT32_MAX); }
  template <class T>
  T* address() {
    return reinterpret_cast<T*>((uintptr_t)integer(0, INT64_MAX));
  }
  float real() {
    PyObject* o = next();
    if (!PyFloat_Check(o) && !PyLong_Check(o)) {
      ok = false;
      return 0.f;
    }
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  // the pool (its address) and its device, which has to be the current one
  const mla_paged_cache* pool() {
    const auto* c = address<const mla_paged_cache>();
    dev = int32();
    if (!ok || dev < 0 || c10::cuda::current_device() != dev) ok = false;
    return c;
  }
  const int32_t* table(int64_t B, int32_t* width) {
    const at::Tensor* t = tensor(at::kInt);
    if (!t || t->dim() != 2 || t->size(0) != B || t->size(1) > INT32_MAX || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    *width = (int32_t)t->size(1);
    return static_cast<const int32_t*>(t->const_data_ptr());
  }
  uint32_t* status() {
    if (none()) return nullptr;
    const at::Tensor* t = dense(at::kInt, {1});
    return ok ? static_cast<uint32_t*>(t->data_ptr()) : nullptr;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

template <class T = int32_t>
const T* at_of(const at::Tensor* t) {
  return static_cast<const T*>(t->const_data_ptr());
}

PyObject* pair(const at::Tensor& x, const at::Tensor& y) {
  PyObject* p = x.defined() ? THPVariable_Wrap(x) : (Py_INCREF(Py_None), Py_None);
  PyObject* q = y.defined() ? THPVariable_Wrap(y) : (Py_INCREF(Py_None), Py_None);
  PyObject* r = p && q ? PyTuple_Pack(2, p, q) : nullptr;
  Py_XDECREF(p);
  Py_XDECREF(q);
  return r;
}
PyObject* answer(mla_status st, const at::Tensor& x, const at::Tensor& y) {
  return st == MLA_OK ? pair(x, y) : PyLong_FromLong(st);
}

// ----------------------------------------------------------------- calls

// (pool, device, pos, table, kv_a, norm_weight, eps, rotary, rotary's device, end_pos, q, q_nope, q_pe, status)
PyObject* append_rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{args, n};
  const mla_paged_cache* pool = a.pool();
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor* pos = a.tensor(at::kInt);
  if (!a.ok || pos->dim() != 2 || !pos->is_contiguous() || pos->size(0) < 1 || pos->size(1) < 1 || pos->numel() > INT32_MAX)
    Py_RETURN_NONE;
  const int64_t B = pos->size(0), s = pos->size(1);
  int32_t width = 0;
  const int32_t* table = a.table(B, &width);
  const at::Tensor* kv = a.rows(at::kBFloat16, {B, s, 576});
  const bool f32 = a.i < n && THPVariable_Check(args[a.i]) && THPVariable_Unpack(args[a.i]).scalar_type() == at::kFloat;
  const at::Tensor* norm = a.dense(f32 ? at::kFloat : at::kBFloat16, {512});
  const float eps = a.real();
  const mla_rotary* rotary = a.address<const mla_rotary>();
  if (a.int32() != a.dev) a.ok = false;
  const at::Tensor* end = a.dense(at::kInt, {B});
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor* q = nullptr;
  at::Tensor nope, pe;
  int64_t H = 0;
  if (!a.none()) {
    q = a.tensor(at::kBFloat16);
    if (!a.ok || q->dim() != 4) Py_RETURN_NONE;
    H = q->size(2);
    if (q->size(0) != B || q->size(1) != s || q->size(3) != 192 || q->stride(3) != 1 || H < 1 || H > 128) Py_RETURN_NONE;
    nope = a.output(at::kBFloat16, {B, s, H, 128});
    pe = a.output(at::kBFloat16, {B, s, H, 64});
  } else if (!(a.none() && a.none())) {
    Py_RETURN_NONE;
  }
  uint32_t* status = a.status();
  if (!a.ok || a.i != n) Py_RETURN_NONE;
  const mla_status st = lib.append_rotary(
      pool, table, width, kv->const_data_ptr(), kv->stride(0), kv->stride(1), norm->const_data_ptr(), f32, eps, rotary, at_of(pos),
      at_of(end), (int32_t)B, (int32_t)s, q ? q->const_data_ptr() : nullptr, q ? q->stride(0) : 0, q ? q->stride(1) : 0,
      q ? q->stride(2) : 0, (int32_t)H, q ? nope.data_ptr() : nullptr, q ? pe.data_ptr() : nullptr, status, a.stream());
  return answer(st, nope, pe);
  END_HANDLE_TH_ERRORS
}

// (pool, device, offsets, table, total, first, kv, pe, status)
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{args, n};
  const mla_paged_cache* pool = a.pool();
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor* off = a.tensor(at::kInt);
  if (!a.ok || off->dim() != 1 || !off->is_contiguous() || off->numel() < 2 || off->numel() > INT32_MAX) Py_RETURN_NONE;
  const int64_t B = off->numel() - 1;
  int32_t width = 0;
  const int32_t* table = a.table(B, &width);
  const int64_t total = a.integer(0, INT32_MAX);
  const at::Tensor* first = nullptr;
  if (!a.none()) first = a.dense(at::kInt, {B});
  if (!a.ok) Py_RETURN_NONE;
  at::Tensor out[2];
  for (int k = 0; k < 2; ++k) {
    const int64_t cols = k ? 64 : 512;
    if (a.none()) {
      out[k] = a.make(at::kBFloat16, {total, cols});
    } else {
      const at::Tensor* t = a.rows(at::kBFloat16, {total, cols});
      if (!a.ok) Py_RETURN_NONE;
      out[k] = *t;
    }
  }
  uint32_t* status = a.status();
  if (!a.ok || a.i != n) Py_RETURN_NONE;
  const mla_status st = lib.read(pool, table, width, at_of(off), first ? at_of(first) : nullptr, (int32_t)B, (int32_t)total,
                                 out[0].data_ptr(), out[0].stride(0), out[1].data_ptr(), out[1].stride(0), status, a.stream());
  return answer(st, out[0], out[1]);
  END_HANDLE_TH_ERRORS
}

// (pool, device, q_latent, table, q_pe, end_pos, max_end_pos, softmax_scale, window, sinks, out, lse, want_lse, workspace)
PyObject* decode_window(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{args, n};
  const mla_paged_cache* pool = a.pool();
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor* ql = a.tensor(at::kBFloat16);
  if (!a.ok || ql->dim() != 4 || !ql->is_contiguous() || ql->size(3) != 512) Py_RETURN_NONE;
  const int64_t B = ql->size(0), s = ql->size(1), H = ql->size(2);
  if (B < 1 || B > 65535 || s < 1 || s > 1024 || H < 1 || H > 128) Py_RETURN_NONE;
  int32_t width = 0;
  const int32_t* table = a.table(B, &width);
  const at::Tensor* qp = a.dense(at::kBFloat16, {B, s, H, 64});
  const at::Tensor* end = a.dense(at::kInt, {B});
  const int32_t max_end = a.int32();
  const float scale = a.real();
  const int32_t window = a.int32(), sinks = a.int32();
  if (!a.ok) Py_RETURN_NONE;
  at::Tensor out = a.output(at::kBFloat16, {B, s, H, 512}), lse, workspace;
  const bool lse_given = a.i < n && args[a.i] != Py_None;
  int asked = 1;
  if (!lse_given && a.i + 1 < n && (asked = PyObject_IsTrue(args[a.i + 1])) < 0) {   // (the binding says what is wrong)
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const bool want = asked != 0;
  if (want)
    lse = a.output(at::kFloat, {B, s, H});
  else
    a.next();
  a.next();   // want_lse
  if (!a.ok) Py_RETURN_NONE;
  if (a.none()) {
    const size_t bytes = lib.window_workspace_size((int32_t)B, (int32_t)s, (int32_t)H);
    if (!bytes) Py_RETURN_NONE;
    workspace = a.make(at::kByte, {(int64_t)bytes});
  } else {
    const at::Tensor* t = a.tensor(at::kByte);
    if (!a.ok || t->dim() != 1 || !t->is_contiguous()) Py_RETURN_NONE;
    workspace = *t;
  }
  if (!a.ok || a.i != n) Py_RETURN_NONE;
  const mla_status st = lib.decode_window(pool, table, width, ql->const_data_ptr(), qp->const_data_ptr(), at_of(end), max_end,
                                          (int32_t)B, (int32_t)s, (int32_t)H, scale, window, sinks, out.data_ptr(),
                                          want ? static_cast<float*>(lse.data_ptr()) : nullptr, workspace.data_ptr(),
                                          (size_t)workspace.numel(), a.stream());
  return answer(st, out, lse);
  END_HANDLE_TH_ERRORS
}

// (addresses of mla_paged_append_rotary, mla_paged_read, mla_paged_decode_window, mla_paged_window_workspace_size)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  Library l;
  l.append_rotary = reinterpret_cast<decltype(l.append_rotary)>(a.address<void>());
  l.read = reinterpret_cast<decltype(l.read)>(a.address<void>());
  l.decode_window = reinterpret_cast<decltype(l.decode_window)>(a.address<void>());
  l.window_workspace_size = reinterpret_cast<decltype(l.window_workspace_size)>(a.address<void>());
  if (!a.ok || !l.append_rotary || !l.read || !l.decode_window || !l.window_workspace_size) {
    PyErr_SetString(PyExc_ValueError, "bind: four addresses");
    return nullptr;
  }
  lib = l;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"append_rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_rotary)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"decode_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_window)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_native() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", MLA_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}

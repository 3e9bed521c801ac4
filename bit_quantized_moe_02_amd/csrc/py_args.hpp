// Looks over the tensors of a call from Python and hands their addresses and
// strides on (py_attn.cpp, py_step.cpp).
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/qmoe_step.h"

#define FAST(f) (PyCFunction)(void (*)(void)) f, METH_FASTCALL, nullptr

namespace {

struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
};

// 16-bit row types
inline int row_type(PyObject* o) {
  if (!THPVariable_Check(o)) return -1;
  const auto t = THPVariable_Unpack(o).scalar_type();
  return t == at::kBFloat16 ? MOE_DT_BF16 : t == at::kHalf ? MOE_DT_F16 : -1;
}

inline bool here(const at::Tensor& t, int64_t dev) { return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev; }

// A row tensor [>= n, heads, dim] on device `dev`, its heads back to back.
inline bool rows(PyObject* o, int64_t heads, int64_t dim, int64_t n, int dtype, int64_t dev, Rows* r) {
  if (row_type(o) != dtype) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!here(t, dev) || t.dim() != 3) return false;
  const auto size = t.sizes(), stride = t.strides();
  if (size[0] < n || size[1] != heads || size[2] != dim || stride[2] != 1 || (stride[1] != dim && heads != 1)) return false;
  r->p = t.data_ptr();
  r->stride = size[0] > 1 ? stride[0] : heads * dim;
  return true;
}

// Heads of a row tensor, 0 for others (which rows() then refuses).
inline int64_t heads_of(PyObject* o) {
  if (!THPVariable_Check(o)) return 0;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.dim() == 3 ? t.size(1) : 0;
}

// A contiguous tensor of at least n elements; its address and size.
inline bool vec(PyObject* o, at::ScalarType type, int64_t n, int64_t dev, void** p, int64_t* numel = nullptr) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!here(t, dev) || t.scalar_type() != type || !t.is_contiguous() || t.numel() < n) return false;
  *p = t.data_ptr();
  if (numel) *numel = t.numel();
  return true;
}

inline bool vec_or_none(PyObject* o, at::ScalarType type, int64_t n, int64_t dev, void** p) {
  return o == Py_None || vec(o, type, n, dev, p);
}

// Numbers and addresses among the arguments; a Python error is left set.
struct Args {
  PyObject* const* a;
  int64_t num(int i) const { return PyLong_AsLongLong(a[i]); }
  void* addr(int i) const { return PyLong_AsVoidPtr(a[i]); }
};

inline PyObject* refused() { return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1); }

template <typename F>
PyObject* call(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f(Args{a});
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The library's call without the interpreter's lock.
template <typename F>
PyObject* run(F f) {
  if (PyErr_Occurred()) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

}  // namespace

// of py_step.cpp
PyObject* step_use(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* step_norm(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* step_linear(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* step_resize(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* step_fork(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* step_compact(PyObject*, PyObject* const*, Py_ssize_t);

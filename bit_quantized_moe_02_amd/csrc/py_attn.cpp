// Arguments of the attention calls from Python: looks over the tensors of a
// call and hands their addresses and strides to the library.  One call of a
// small step is a few microseconds on the GPU, and looking at each of its
// tensors through Python took as long (append of one token 7.4 us a call on
// the host, of which the library's launch 3.0).
//
// Each function returns the library's code, or -1 when a tensor is not what
// the call needs; the caller finds out which and says so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/qmoe_attn.h"

namespace {

// the library's functions (the library itself is loaded by the caller)
decltype(&moe_kv_append) p_append;
decltype(&moe_kv_read) p_read;
decltype(&moe_attn_decode) p_decode;
decltype(&moe_attn_prefill) p_prefill;

struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
};

// 16-bit row types
int row_type(PyObject* o) {
  if (!THPVariable_Check(o)) return -1;
  const auto t = THPVariable_Unpack(o).scalar_type();
  return t == at::kBFloat16 ? MOE_DT_BF16 : t == at::kHalf ? MOE_DT_F16 : -1;
}

bool here(const at::Tensor& t, int64_t dev) { return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev; }

// A row tensor [>= n, heads, dim] on device `dev`, its heads back to back.
bool rows(PyObject* o, int64_t heads, int64_t dim, int64_t n, int dtype, int64_t dev, Rows* r) {
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
int64_t heads_of(PyObject* o) {
  if (!THPVariable_Check(o)) return 0;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.dim() == 3 ? t.size(1) : 0;
}

// A contiguous tensor of at least n elements; its address and size.
bool vec(PyObject* o, at::ScalarType type, int64_t n, int64_t dev, void** p, int64_t* numel = nullptr) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!here(t, dev) || t.scalar_type() != type || !t.is_contiguous() || t.numel() < n) return false;
  *p = t.data_ptr();
  if (numel) *numel = t.numel();
  return true;
}

bool vec_or_none(PyObject* o, at::ScalarType type, int64_t n, int64_t dev, void** p) {
  return o == Py_None || vec(o, type, n, dev, p);
}

// Numbers and addresses among the arguments; a Python error is left set.
struct Args {
  PyObject* const* a;
  int64_t num(int i) const { return PyLong_AsLongLong(a[i]); }
  void* addr(int i) const { return PyLong_AsVoidPtr(a[i]); }
};

PyObject* refused() { return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1); }

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

// use(append, read, decode, prefill): addresses of the library's functions
PyObject* use(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 4, [](Args a) -> PyObject* {
    p_append = reinterpret_cast<decltype(p_append)>(a.addr(0));
    p_read = reinterpret_cast<decltype(p_read)>(a.addr(1));
    p_decode = reinterpret_cast<decltype(p_decode)>(a.addr(2));
    p_prefill = reinterpret_cast<decltype(p_prefill)>(a.addr(3));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  });
}

// append(cache, batch, rope, heads, dim, rows, device, stream, k, v, q, q_out, k_out)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 13, [](Args a) -> PyObject* {
    const int64_t heads = a.num(3), dim = a.num(4), r = a.num(5), dev = a.num(6);
    const int dt = row_type(a.a[8]);
    Rows k, v, q, qo, ko;
    int64_t hq = 0;
    if (dt < 0 || !rows(a.a[8], heads, dim, r, dt, dev, &k) || !rows(a.a[9], heads, dim, r, dt, dev, &v)) return refused();
    if (a.a[10] != Py_None) {
      hq = heads_of(a.a[10]);
      if (!rows(a.a[10], hq, dim, r, dt, dev, &q) || !rows(a.a[11], hq, dim, r, dt, dev, &qo)) return refused();
    }
    if (a.a[12] != Py_None && !rows(a.a[12], heads, dim, r, dt, dev, &ko)) return refused();
    const auto cache = (const moe_kv_cache*)a.addr(0);
    const auto batch = (const moe_kv_batch*)a.addr(1);
    const auto rope = (const moe_rope*)a.addr(2);
    void* const stream = a.addr(7);
    return run([&] {
      return p_append(cache, batch, rope, dt, q.p, q.stride, (int32_t)hq, k.p, k.stride, v.p, v.stride, qo.p, qo.stride, ko.p,
                      ko.stride, stream);
    });
  });
}

// read(cache, batch, heads, dim, rows, device, stream, k_out, v_out)
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 9, [](Args a) -> PyObject* {
    const int64_t heads = a.num(2), dim = a.num(3), r = a.num(4), dev = a.num(5);
    const int dt = row_type(a.a[7]);
    Rows k, v;
    if (dt < 0 || !rows(a.a[7], heads, dim, r, dt, dev, &k) || !rows(a.a[8], heads, dim, r, dt, dev, &v)) return refused();
    const auto cache = (const moe_kv_cache*)a.addr(0);
    const auto batch = (const moe_kv_batch*)a.addr(1);
    void* const stream = a.addr(6);
    return run([&] { return p_read(cache, batch, dt, k.p, k.stride, v.p, v.stride, stream); });
  });
}

// decode(cache, batch, dim, rows, device, stream, q, out, ws, scale, lse)
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 11, [](Args a) -> PyObject* {
    const int64_t dim = a.num(2), r = a.num(3), dev = a.num(4), hq = heads_of(a.a[6]);
    const int dt = row_type(a.a[6]);
    Rows q, out;
    void *ws = nullptr, *lse = nullptr;
    int64_t ws_bytes = 0;
    if (dt < 0 || !rows(a.a[6], hq, dim, r, dt, dev, &q) || !rows(a.a[7], hq, dim, r, dt, dev, &out) ||
        !vec(a.a[8], at::kByte, 0, dev, &ws, &ws_bytes) || !vec_or_none(a.a[10], at::kFloat, r * hq, dev, &lse))
      return refused();
    const auto cache = (const moe_kv_cache*)a.addr(0);
    const auto batch = (const moe_kv_batch*)a.addr(1);
    void* const stream = a.addr(5);
    const float scale = (float)PyFloat_AsDouble(a.a[9]);
    return run([&] {
      return p_decode(cache, batch, dt, q.p, q.stride, (int32_t)hq, scale, out.p, out.stride, (float*)lse, ws, (size_t)ws_bytes,
                      stream);
    });
  });
}

// prefill(device, stream, q, k, v, cu_q, cu_k, max_q, out, ws, scale, causal, lse)
PyObject* prefill(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 13, [](Args a) -> PyObject* {
    const int64_t dev = a.num(0), max_q = a.num(7), hq = heads_of(a.a[2]), hk = heads_of(a.a[3]);
    const int dt = row_type(a.a[2]);
    if (dt < 0 || hq == 0 || hk == 0) return refused();
    const at::Tensor &tq = THPVariable_Unpack(a.a[2]), &tk = THPVariable_Unpack(a.a[3]);
    const int64_t nq = tq.size(0), nk = tk.size(0), dim = tq.size(2);
    Rows q, k, v, out;
    void *cu_q = nullptr, *cu_k = nullptr, *ws = nullptr, *lse = nullptr;
    int64_t n_cu = 0, ws_bytes = 0;
    constexpr int64_t most = 0x7FFFFFFF;    // (the library refuses less than that by itself)
    if (!rows(a.a[2], hq, dim, nq, dt, dev, &q) || !rows(a.a[3], hk, dim, nk, dt, dev, &k) ||
        !rows(a.a[4], hk, dim, nk, dt, dev, &v) || !rows(a.a[8], hq, dim, nq, dt, dev, &out) ||
        !vec(a.a[5], at::kInt, 2, dev, &cu_q, &n_cu) || !vec(a.a[6], at::kInt, n_cu, dev, &cu_k) ||
        !vec(a.a[9], at::kByte, 0, dev, &ws, &ws_bytes) || !vec_or_none(a.a[12], at::kFloat, nq * hq, dev, &lse) ||
        max_q < 1 || max_q > most || nq > most || nk > most || n_cu > most || hq > most || hk > most || dim > most)
      return refused();
    const moe_packed p{(int32_t)(n_cu - 1), (int32_t)nq, (int32_t)nk, (int32_t)max_q, (const int32_t*)cu_q,
                       (const int32_t*)cu_k, (int32_t)hq, (int32_t)hk, (int32_t)dim};
    void* const stream = a.addr(1);
    const float scale = (float)PyFloat_AsDouble(a.a[10]);
    const int causal = PyObject_IsTrue(a.a[11]);
    return run([&] {
      return p_prefill(&p, dt, q.p, q.stride, k.p, k.stride, v.p, v.stride, scale, causal, out.p, out.stride, (float*)lse, ws,
                       (size_t)ws_bytes, stream);
    });
  });
}

#define FAST(f) (PyCFunction)(void (*)(void)) f, METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"use", FAST(use)},       {"append", FAST(append)},   {"read", FAST(read)},
                         {"decode", FAST(decode)}, {"prefill", FAST(prefill)}, {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_attn", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn() { return PyModule_Create(&module_def); }

// Arguments of the norm, the 4-bit products and the page calls from Python, as
// py_attn.cpp does it for the attention calls: each function returns the
// library's code, or -1 when a tensor is not what the call needs.
#include "py_args.hpp"

namespace {

// the library's functions (the library itself is loaded by the caller)
decltype(&moe_rms_norm) p_norm;
decltype(&moe_linear) p_linear;
decltype(&moe_kv_resize) p_resize;
decltype(&moe_kv_fork) p_fork;
decltype(&moe_kv_compact) p_compact;

int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    case at::kFloat: return MOE_DT_F32;
    case at::kChar: return MOE_DT_I8;
    default: return -1;
  }
}

constexpr int64_t kMost = 0x7FFFFFFF;    // (the library refuses less than that by itself)

// Rows of vectors: a tensor [rows, cols] or [rows, heads, cols], a row's values back to back.
struct Vectors {
  void* p = nullptr;
  int64_t stride = 0, rows = 0, heads = 0, cols = 0;
  int type = -1;
};

bool vectors(PyObject* o, int64_t dev, Vectors* v) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!here(t, dev) || t.dim() < 2 || t.dim() > 3) return false;
  const auto size = t.sizes(), stride = t.strides();
  const int last = (int)t.dim() - 1;
  v->type = type_of(t);
  v->rows = size[0];
  v->heads = last == 2 ? size[1] : 1;
  v->cols = size[last];
  if (v->type < 0 || v->rows > kMost || v->heads > kMost || v->cols > kMost) return false;
  if (stride[last] != 1 && v->cols > 1) return false;
  if (last == 2 && stride[1] != v->cols && v->heads > 1) return false;
  v->p = t.data_ptr();
  v->stride = v->rows > 1 ? stride[0] : v->heads * v->cols;
  return true;
}

// The same shape as `like`.
bool vectors_as(PyObject* o, const Vectors& like, int64_t dev, Vectors* v) {
  return vectors(o, dev, v) && v->rows == like.rows && v->heads == like.heads && v->cols == like.cols;
}

// fp32 [groups, at least rows]
bool scales_of(PyObject* o, int64_t groups, int64_t rows, int64_t dev, float** p, int64_t* stride) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!here(t, dev) || t.scalar_type() != at::kFloat || t.dim() != 2) return false;
  if (t.size(0) != groups || t.size(1) < rows || (t.stride(1) != 1 && t.size(1) > 1)) return false;
  *p = (float*)t.data_ptr();
  *stride = groups > 1 ? t.stride(0) : t.size(1);
  return true;
}

// The storage holds the last group's scales up to the next multiple of 4 rows.
bool whole_scales(PyObject* o, int64_t groups, int64_t rows, int64_t stride) {
  const at::Tensor& t = THPVariable_Unpack(o);
  return (t.storage_offset() + (groups - 1) * stride + (rows + 3) / 4 * 4) * 4 <= (int64_t)t.storage().nbytes();
}

}  // namespace

// step_use(norm, linear, resize, fork, compact): addresses of the library's functions
PyObject* step_use(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 5, [](Args a) -> PyObject* {
    p_norm = reinterpret_cast<decltype(p_norm)>(a.addr(0));
    p_linear = reinterpret_cast<decltype(p_linear)>(a.addr(1));
    p_resize = reinterpret_cast<decltype(p_resize)>(a.addr(2));
    p_fork = reinterpret_cast<decltype(p_fork)>(a.addr(3));
    p_compact = reinterpret_cast<decltype(p_compact)>(a.addr(4));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  });
}

// step_norm(device, stream, x, out, weight, eps, residual, sum, codes, scales, group)
PyObject* step_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 11, [](Args a) -> PyObject* {
    const int64_t dev = a.num(0), group = a.num(10);
    Vectors x, out, res, sum, codes;
    if (!vectors(a.a[2], dev, &x) || (a.a[3] != Py_None && !vectors_as(a.a[3], x, dev, &out)) ||
        (a.a[6] != Py_None && !vectors_as(a.a[6], x, dev, &res)) ||
        (a.a[7] != Py_None && (!vectors_as(a.a[7], x, dev, &sum) || sum.type != res.type)) ||
        (a.a[8] != Py_None && (!vectors_as(a.a[8], x, dev, &codes) || codes.type != MOE_DT_I8)) || group < 0 || group > kMost)
      return refused();
    moe_norm p{};
    if (a.a[4] != Py_None) {
      if (!THPVariable_Check(a.a[4])) return refused();
      const at::Tensor& w = THPVariable_Unpack(a.a[4]);
      if (!here(w, dev) || !w.is_contiguous() || w.dim() != 1 || w.numel() != x.cols || type_of(w) < 0) return refused();
      p.weight = w.data_ptr();
      p.weight_dtype = type_of(w);
    }
    if (a.a[9] != Py_None) {
      const int64_t groups = x.heads * (group ? (x.cols + group - 1) / group : 1);
      if (!scales_of(a.a[9], groups, x.rows, dev, &p.scales, &p.scale_stride)) return refused();
    }
    p.rows = (int32_t)x.rows;
    p.heads = (int32_t)x.heads;
    p.cols = (int32_t)x.cols;
    p.x_dtype = x.type;
    p.x = x.p;
    p.x_stride = x.stride;
    p.residual_dtype = res.type;
    p.residual = res.p;
    p.residual_stride = res.stride;
    p.sum = sum.p;
    p.sum_stride = sum.stride;
    p.eps = (float)PyFloat_AsDouble(a.a[5]);
    p.out_dtype = out.type;
    p.out = out.p;
    p.out_stride = out.stride;
    p.codes = (int8_t*)codes.p;
    p.codes_stride = codes.stride;
    p.group = (int32_t)group;
    void* const stream = a.addr(1);
    return run([&] { return p_norm(&p, stream); });
  });
}

// step_linear(weights, n, k, device, stream, x, y, x_scales, x_group)
PyObject* step_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 9, [](Args a) -> PyObject* {
    const int64_t wn = a.num(1), wk = a.num(2), dev = a.num(3), group = a.num(8);
    Vectors x, y;
    if (!vectors(a.a[5], dev, &x) || !vectors(a.a[6], dev, &y) || x.heads * x.cols != wk || y.heads * y.cols != wn ||
        y.rows != x.rows || group < 0 || group > kMost)
      return refused();
    float* scales = nullptr;
    int64_t scale_stride = 0;
    const int64_t groups = group ? (wk + group - 1) / group : 1;
    if (a.a[7] != Py_None && (!scales_of(a.a[7], groups, x.rows, dev, &scales, &scale_stride) ||
                              (group && !whole_scales(a.a[7], groups, x.rows, scale_stride))))
      return refused();
    const auto w = (const moe_linear_weights*)a.addr(0);
    void* const stream = a.addr(4);
    return run([&] {
      return p_linear(w, (int32_t)x.rows, x.type, x.p, x.stride, scales, scale_stride, (int32_t)group, y.type, y.p, y.stride, stream);
    });
  });
}

// step_resize(pool, tables, seqs, device, stream, new_lens, missing)
PyObject* step_resize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 7, [](Args a) -> PyObject* {
    const int64_t seqs = a.num(2), dev = a.num(3);
    void *lens = nullptr, *missing = nullptr;
    if (!vec(a.a[5], at::kInt, seqs, dev, &lens) || !vec_or_none(a.a[6], at::kInt, 1, dev, &missing)) return refused();
    const auto pool = (const moe_kv_pool*)a.addr(0);
    const auto tables = (const moe_kv_tables*)a.addr(1);
    void* const stream = a.addr(4);
    return run([&] { return p_resize(pool, tables, (const int32_t*)lens, (int32_t*)missing, stream); });
  });
}

// step_fork(pool, tables, seqs, device, stream, from, missing, ws)
PyObject* step_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 8, [](Args a) -> PyObject* {
    const int64_t seqs = a.num(2), dev = a.num(3);
    void *from = nullptr, *missing = nullptr, *ws = nullptr;
    int64_t ws_bytes = 0;
    if (!vec(a.a[5], at::kInt, seqs, dev, &from) || !vec_or_none(a.a[6], at::kInt, 1, dev, &missing) ||
        !vec(a.a[7], at::kByte, 0, dev, &ws, &ws_bytes))
      return refused();
    const auto pool = (const moe_kv_pool*)a.addr(0);
    const auto tables = (const moe_kv_tables*)a.addr(1);
    void* const stream = a.addr(4);
    return run([&] { return p_fork(pool, tables, (const int32_t*)from, (int32_t*)missing, ws, (size_t)ws_bytes, stream); });
  });
}

// step_compact(pool, tables, device, stream, held, ws)
PyObject* step_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 6, [](Args a) -> PyObject* {
    const int64_t dev = a.num(2);
    void *held = nullptr, *ws = nullptr;
    int64_t ws_bytes = 0;
    if (!vec_or_none(a.a[4], at::kInt, 1, dev, &held) || !vec(a.a[5], at::kByte, 0, dev, &ws, &ws_bytes)) return refused();
    const auto pool = (const moe_kv_pool*)a.addr(0);
    const auto tables = (const moe_kv_tables*)a.addr(1);
    void* const stream = a.addr(3);
    return run([&] { return p_compact(pool, tables, (int32_t*)held, ws, (size_t)ws_bytes, stream); });
  });
}

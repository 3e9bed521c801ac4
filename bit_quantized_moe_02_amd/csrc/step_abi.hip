// C ABI of the calls around attention and the experts (include/qmoe_step.h):
// argument checks, workspace sizes and launches.  (The host-only calls are in
// host_linear.cpp.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "../../include/qmoe_step.h"
#include "k_step.h"
#include "qmoe_internal.h"

using namespace qmoe;

namespace {

constexpr int64_t kMaxRows = 1 << 24;
constexpr int64_t kMaxProductRows = 1 << 20;     // (at 64 to a workgroup they fit the grid's second dimension)
constexpr int64_t kMaxStride = 1 << 24;
constexpr int64_t kMaxVectors = (1 << 24) - 1;
constexpr int64_t kMaxThreads = (1ll << 32) - 1;  // of a launch
constexpr int kMaxCaches = 256;
constexpr int kMaxSeqs = 4096;                   // two numbers a row in LDS

bool aligned(const void* p, uintptr_t by) { return ((uintptr_t)p & (by - 1)) == 0; }

int bad(const char* who, const std::string& what) { return fail(MOE_ERR_INVALID_ARG, std::string(who) + ": " + what); }

int done(const char* who, hipError_t e) {
  return e == hipSuccess ? MOE_OK : fail(MOE_ERR_HIP, std::string(who) + ": " + hipGetErrorString(e));
}

// Compute units of the current device (asked for once per device).
int n_cus() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  cus = known[dev].load(std::memory_order_relaxed);
  if (cus > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
  known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

bool float_type(int t) { return t == MOE_DT_BF16 || t == MOE_DT_F16 || t == MOE_DT_F32; }

// A row tensor of `width` elements a row.
int check_rows(const char* who, const char* name, const void* p, int64_t stride, int64_t width) {
  if (!p) return bad(who, std::string(name) + " is NULL");
  if (!aligned(p, 16)) return bad(who, std::string(name) + " must be 16-byte aligned");
  if (stride < width || stride % 8 != 0 || stride > kMaxStride)
    return bad(who, std::string(name) + "'s stride must be a multiple of 8, at least a row's length, at most 2^24");
  return MOE_OK;
}

// In place means the very same rows: same type and stride.
int check_place(const char* who, const char* out, const void* o, int ot, int64_t os, const char* in, const void* i, int it,
                int64_t is) {
  if (o && o == i && (ot != it || os != is)) return bad(who, std::string(out) + " in place of " + in + " needs its type and stride");
  return MOE_OK;
}

}  // namespace

extern "C" int moe_rms_norm(const moe_norm* p, void* stream) {
  clear_error();
  static const char* who = "moe_rms_norm";
  if (!p) return bad(who, "the description is NULL");
  if (p->rows < 0 || p->rows > kMaxRows) return bad(who, "need 0 <= rows <= 2^24");
  if (p->cols < 8 || p->cols > 16384 || p->cols % 8 != 0) return bad(who, "cols must be a multiple of 8 in [8, 16384]");
  if (p->heads < 1 || p->heads > 4096 || (int64_t)p->heads * p->rows > kMaxVectors ||
      (int64_t)p->heads * p->rows * norm_threads(p->cols) > kMaxThreads)
    return bad(who, "need 1 <= heads <= 4096, rows * heads < 2^24 (cols > 2048: 2^23, cols > 4096: 2^22)");
  if (!(p->eps >= 0) || !isfinite(p->eps)) return bad(who, "eps must be finite and not negative");
  if (!float_type(p->x_dtype) || (p->residual && !float_type(p->residual_dtype)) || (p->weight && !float_type(p->weight_dtype)) ||
      (p->out && !float_type(p->out_dtype)))
    return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": unknown type");
  if (p->rows == 0) return MOE_OK;
  const int64_t width = (int64_t)p->heads * p->cols;
  int rc = check_rows(who, "x", p->x, p->x_stride, width);
  if (rc != MOE_OK) return rc;
  if (p->residual && (rc = check_rows(who, "residual", p->residual, p->residual_stride, width)) != MOE_OK) return rc;
  if (!p->out && !p->codes && !p->sum) return bad(who, "no output is wanted");
  if (p->sum && !p->residual) return bad(who, "sum needs a residual");
  if (p->sum && (rc = check_rows(who, "sum", p->sum, p->sum_stride, width)) != MOE_OK) return rc;
  if (p->out && (rc = check_rows(who, "out", p->out, p->out_stride, width)) != MOE_OK) return rc;
  if (!aligned(p->weight, 16)) return bad(who, "weight must be 16-byte aligned");
  if ((p->codes == nullptr) != (p->scales == nullptr)) return bad(who, "codes and scales belong together");
  if (p->codes) {
    if ((rc = check_rows(who, "codes", p->codes, p->codes_stride, width)) != MOE_OK) return rc;
    if (p->group != 0 && p->group != 128) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": group must be 128 or 0");
    if (!aligned(p->scales, 16)) return bad(who, "scales must be 16-byte aligned");
    if (p->scale_stride < p->rows || p->scale_stride % 4 != 0 || p->scale_stride < 4 || p->scale_stride > (1 << 28))
      return bad(who, "scale_stride must be a multiple of 4, at least rows, at most 2^28");
  }
  if (p->out && (p->out == p->sum || (const void*)p->out == (const void*)p->codes)) return bad(who, "outputs must not overlap");
  if (p->codes && (const void*)p->codes == (const void*)p->sum) return bad(who, "outputs must not overlap");
  if (p->codes && ((const void*)p->codes == p->x || (const void*)p->codes == p->residual)) return bad(who, "codes must not overlap inputs");
  if ((rc = check_place(who, "sum", p->sum, p->residual_dtype, p->sum_stride, "x", p->x, p->x_dtype, p->x_stride)) != MOE_OK) return rc;
  if ((rc = check_place(who, "sum", p->sum, p->residual_dtype, p->sum_stride, "residual", p->residual, p->residual_dtype,
                        p->residual_stride)) != MOE_OK)
    return rc;
  if ((rc = check_place(who, "out", p->out, p->out_dtype, p->out_stride, "x", p->x, p->x_dtype, p->x_stride)) != MOE_OK) return rc;
  if ((rc = check_place(who, "out", p->out, p->out_dtype, p->out_stride, "residual", p->residual, p->residual_dtype,
                        p->residual_stride)) != MOE_OK)
    return rc;
  NormArgs a{};
  a.x = p->x;
  a.res = p->residual;
  a.w = p->weight;
  a.sum = p->sum;
  a.out = p->out;
  a.codes = p->codes;
  a.scales = p->scales;
  a.xs = p->x_stride;
  a.rs = p->residual_stride;
  a.ss = p->sum_stride;
  a.os = p->out_stride;
  a.cs = p->codes_stride;
  a.scs = p->scale_stride;
  a.rows = p->rows;
  a.per_col = 1.0 / p->cols;
  a.heads = p->heads;
  a.cols = p->cols;
  a.group = p->group;
  a.xt = p->x_dtype;
  a.rt = p->residual_dtype;
  a.wt = p->weight_dtype;
  a.ot = p->out_dtype;
  a.eps = p->eps;
  return done(who, launch_norm(a, (hipStream_t)stream));
}

extern "C" int moe_linear(const moe_linear_weights* w, int32_t rows, int x_dtype, const void* x, int64_t x_stride,
                          const float* x_scales, int64_t scale_stride, int32_t x_group, int y_dtype, void* y, int64_t y_stride,
                          void* stream) {
  clear_error();
  static const char* who = "moe_linear";
  if (!w) return bad(who, "the weights are NULL");
  if (moe_linear_packed_bytes(w->n, w->k, w->group, w->with_zeros) == 0)
    return bad(who, "n must be in [1, 2^24], k a multiple of 8 in [8, 2^20], group 32, 64 or 128");
  if (!w->packed || !aligned(w->packed, 16)) return bad(who, "packed must be 16-byte aligned memory");
  if (!aligned(w->bias, 4)) return bad(who, "bias must be 4-byte aligned");
  if (rows < 0 || rows > kMaxProductRows) return bad(who, "need 0 <= rows <= 2^20");
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F16 && x_dtype != MOE_DT_I8)
    return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": unknown type of x");
  if (!float_type(y_dtype)) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": unknown type of y");
  if (rows == 0) return MOE_OK;
  int rc = check_rows(who, "x", x, x_stride, w->k);
  if (rc != MOE_OK) return rc;
  if (x_dtype == MOE_DT_I8) {
    if (!x_scales || !aligned(x_scales, 16)) return bad(who, "8-bit rows need x_scales, 16-byte aligned");
    if (x_group != 0 && x_group != 128) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": x_group must be 128 or 0");
    if (scale_stride < rows || scale_stride % 4 != 0 || scale_stride < 4 || scale_stride > (1 << 28))
      return bad(who, "scale_stride must be a multiple of 4, at least rows, at most 2^28");
  } else if (x_scales || x_group) {
    return bad(who, "16-bit rows have no scales");
  }
  if (!y || !aligned(y, 16)) return bad(who, "y must be 16-byte aligned memory");
  if (y_stride < w->n || y_stride > kMaxStride) return bad(who, "y_stride must be at least n, at most 2^24");
  if (y == x) return bad(who, "y must not overlap x");
  LinearArgs a{};
  a.w = (const uint8_t*)w->packed;
  a.bias = w->bias;
  a.x = x;
  a.xs = x_scales;
  a.y = y;
  a.x_stride = x_stride;
  a.xs_stride = scale_stride;
  a.y_stride = y_stride;
  a.n = w->n;
  a.k = w->k;
  a.rows = rows;
  a.y_type = y_dtype;
  a.zeros = w->with_zeros != 0;
  a.x_group = x_group;
  return done(who, launch_linear(a, x_dtype, w->group, n_cus(), (hipStream_t)stream));
}

namespace qmoe {

template <int XT>
hipError_t launch_linear_type(const LinearArgs& a, int group, int cus, hipStream_t s);
extern template hipError_t launch_linear_type<MOE_DT_BF16>(const LinearArgs&, int, int, hipStream_t);
extern template hipError_t launch_linear_type<MOE_DT_F16>(const LinearArgs&, int, int, hipStream_t);
extern template hipError_t launch_linear_type<MOE_DT_I8>(const LinearArgs&, int, int, hipStream_t);

hipError_t launch_linear(const LinearArgs& a, int x_type, int group, int cus, hipStream_t s) {
  if (x_type == MOE_DT_BF16) return launch_linear_type<MOE_DT_BF16>(a, group, cus, s);
  if (x_type == MOE_DT_F16) return launch_linear_type<MOE_DT_F16>(a, group, cus, s);
  return launch_linear_type<MOE_DT_I8>(a, group, cus, s);
}

}  // namespace qmoe

namespace {

int check_pages(const char* who, const moe_kv_pool* pool, const moe_kv_tables* t, PagesArgs* a) {
  if (!pool || !t) return bad(who, "pool or tables is NULL");
  if (pool->n_pages < 1 || pool->n_pages > (1 << 29)) return bad(who, "need 1 <= n_pages <= 2^29");
  if (pool->n_caches < 0 || pool->n_caches > kMaxCaches || (pool->n_caches > 0 && !pool->caches))
    return bad(who, "need 0 <= n_caches <= 256, and caches");
  if (!pool->refs || !aligned(pool->refs, 16)) return bad(who, "refs must be 16-byte aligned memory");
  const int page = t->page_tokens;
  if (page < 16 || page > 1024 || (page & (page - 1)) != 0) return bad(who, "page_tokens must be a power of two in [16, 1024]");
  if (t->seqs < 1 || t->seqs > kMaxSeqs || t->pages_per_seq < 1) return bad(who, "need 1 <= seqs <= 4096, pages_per_seq >= 1");
  if ((int64_t)t->pages_per_seq * page > (1 << 30) || (int64_t)t->pages_per_seq * t->seqs > (1 << 30))
    return bad(who, "more than 2^30 positions a sequence, or 2^30 pages of all");
  if (!t->page_table || !aligned(t->page_table, 4) || !t->kv_lens || !aligned(t->kv_lens, 4))
    return bad(who, "page_table and kv_lens must be 4-byte aligned memory");
  if (t->table_stride < t->pages_per_seq) return bad(who, "table_stride must be at least pages_per_seq");
  for (int i = 0; i < pool->n_caches; ++i) {
    const moe_kv_cache& c = pool->caches[i];
    if (c.n_pages != pool->n_pages || c.page_tokens != page) return bad(who, "the caches' n_pages and page_tokens must be the pool's and the tables'");
    if (moe_kv_code_bytes(c.n_pages, c.page_tokens, c.kv_heads, c.head_dim) == 0) return bad(who, "a cache's heads are not valid");
    if (!c.codes || !c.scales || !aligned(c.codes, 16) || !aligned(c.scales, 4))
      return bad(who, "the caches' codes must be 16-byte aligned memory, their scales 4-byte aligned");
  }
  a->refs = pool->refs;
  a->table = t->page_table;
  a->lens = t->kv_lens;
  a->stride = t->table_stride;
  a->n_pages = pool->n_pages;
  a->seqs = t->seqs;
  a->per_seq = t->pages_per_seq;
  a->shift = 0;
  while ((1 << a->shift) < page) ++a->shift;
  return MOE_OK;
}

// The pool's caches in the launches' form.
struct Copies {
  PageCopy c[kMaxCaches / kCachesALaunch] = {};
  explicit Copies(const moe_kv_pool* pool) {
    for (int i = 0; i < pool->n_caches; ++i) {
      const moe_kv_cache& k = pool->caches[i];
      PageCopy& p = c[i / kCachesALaunch];
      const int at = i % kCachesALaunch;
      p.codes[at] = (uint8_t*)k.codes;
      p.scales[at] = k.scales;
      p.heads[at] = k.kv_heads;
      p.block[at] = 32 * k.head_dim;
    }
  }
};

size_t fork_ws(const PagesArgs& a) { return kForkHead + (size_t)a.seqs * sizeof(ForkJob); }
size_t compact_ws(const PagesArgs& a) { return 16 + (size_t)a.n_pages * 12; }

int check_ws(const char* who, const void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned(ws, 16)) return bad(who, "ws must be 16-byte aligned memory");
  if (bytes < need) return fail(MOE_ERR_WORKSPACE, std::string(who) + ": workspace too small (need " + std::to_string(need) + ")");
  return MOE_OK;
}

}  // namespace

extern "C" int moe_kv_resize(const moe_kv_pool* pool, const moe_kv_tables* tables, const int32_t* new_lens, int32_t* missing,
                             void* stream) {
  clear_error();
  static const char* who = "moe_kv_resize";
  PagesArgs a{};
  const int rc = check_pages(who, pool, tables, &a);
  if (rc != MOE_OK) return rc;
  if (!new_lens || !aligned(new_lens, 4) || !aligned(missing, 4)) return bad(who, "new_lens and missing must be 4-byte aligned memory");
  if (new_lens == a.lens) return bad(who, "new_lens must not be kv_lens");
  return done(who, launch_resize(a, new_lens, missing, (hipStream_t)stream));
}

extern "C" size_t moe_kv_fork_workspace_bytes(const moe_kv_pool* pool, const moe_kv_tables* tables) {
  clear_error();
  PagesArgs a{};
  return check_pages("moe_kv_fork_workspace_bytes", pool, tables, &a) == MOE_OK ? fork_ws(a) : 0;
}

extern "C" int moe_kv_fork(const moe_kv_pool* pool, const moe_kv_tables* tables, const int32_t* from, int32_t* missing, void* ws,
                           size_t ws_bytes, void* stream) {
  clear_error();
  static const char* who = "moe_kv_fork";
  PagesArgs a{};
  int rc = check_pages(who, pool, tables, &a);
  if (rc != MOE_OK) return rc;
  if (!from || !aligned(from, 4) || !aligned(missing, 4)) return bad(who, "from and missing must be 4-byte aligned memory");
  if ((rc = check_ws(who, ws, ws_bytes, fork_ws(a))) != MOE_OK) return rc;
  const Copies c(pool);
  return done(who, launch_fork(a, from, missing, ws, c.c, pool->n_caches, n_cus(), (hipStream_t)stream));
}

extern "C" size_t moe_kv_compact_workspace_bytes(const moe_kv_pool* pool, const moe_kv_tables* tables) {
  clear_error();
  PagesArgs a{};
  return check_pages("moe_kv_compact_workspace_bytes", pool, tables, &a) == MOE_OK ? compact_ws(a) : 0;
}

extern "C" int moe_kv_compact(const moe_kv_pool* pool, const moe_kv_tables* tables, int32_t* held, void* ws, size_t ws_bytes,
                              void* stream) {
  clear_error();
  static const char* who = "moe_kv_compact";
  PagesArgs a{};
  int rc = check_pages(who, pool, tables, &a);
  if (rc != MOE_OK) return rc;
  if (!aligned(held, 4)) return bad(who, "held must be 4-byte aligned");
  if ((rc = check_ws(who, ws, ws_bytes, compact_ws(a))) != MOE_OK) return rc;
  const Copies c(pool);
  return done(who, launch_compact(a, held, (int32_t*)ws, c.c, pool->n_caches, n_cus(), (hipStream_t)stream));
}

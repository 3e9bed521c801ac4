// C ABI of the attention calls (include/qmoe_attn.h): argument checks,
// workspace layout and launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "../../include/qmoe_attn.h"
#include "k_attn.h"
#include "qmoe_internal.h"

using namespace qmoe;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = 1 << 24;       // rows of a call
constexpr int64_t kMaxStride = 1 << 24;     // elements: a tile's offsets then fit 32 bits
constexpr int64_t kMaxGrid = (1 << 24) - 1; // workgroups of 256 threads: 32-bit thread numbers
constexpr int64_t kMaxBatch = 1 << 20;
constexpr float kLog2e = 1.4426950408889634f;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int bad(const char* who, const std::string& what) { return fail(MOE_ERR_INVALID_ARG, std::string(who) + ": " + what); }

int hip_fail(const char* who, hipError_t e) {
  return fail(MOE_ERR_HIP, std::string(who) + ": " + hipGetErrorString(e));
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

bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_ok(int p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
bool geometry_ok(int32_t n_pages, int32_t page_tokens, int32_t kv_heads) {
  return n_pages >= 1 && page_ok(page_tokens) && kv_heads >= 1 && kv_heads <= 256;
}

int log2i(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// A row tensor: pointer, alignment, stride.
int check_rows(const char* who, const char* name, const void* p, int64_t stride, int heads, int dim) {
  if (!p) return bad(who, std::string(name) + " is NULL");
  if (!aligned16(p)) return bad(who, std::string(name) + " must be 16-byte aligned");
  if (stride < (int64_t)heads * dim || stride % 8 != 0 || stride > kMaxStride)
    return bad(who, std::string(name) + "'s stride must be a multiple of 8, at least heads * head_dim, at most 2^24");
  return MOE_OK;
}

int check_dtype(const char* who, int dtype) {
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": unknown row type");
  return MOE_OK;
}

int check_cache(const char* who, const moe_kv_cache* c, const moe_kv_batch* b, KvArgs* a) {
  if (!c || !b) return bad(who, "cache or batch is NULL");
  if (!geometry_ok(c->n_pages, c->page_tokens, c->kv_heads))
    return bad(who, "need n_pages >= 1, page_tokens a power of two in [16, 1024], 1 <= kv_heads <= 256");
  if (!dim_ok(c->head_dim)) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": head_dim must be 64, 128 or 256");
  if (!c->codes || !c->scales) return bad(who, "the cache's codes or scales are NULL");
  if (!aligned16(c->codes) || !aligned16(c->scales)) return bad(who, "the cache must be 16-byte aligned");
  if (b->batch < 1 || b->batch > kMaxBatch || b->rows < 1 || b->rows > kMaxRows || b->max_new < 1 || b->pages_per_seq < 1)
    return bad(who, "need batch, rows, max_new and pages_per_seq >= 1, batch <= 2^20, rows <= 2^24");
  if (!b->page_table || !b->kv_lens) return bad(who, "page_table or kv_lens is NULL");
  if (!aligned4(b->page_table) || !aligned4(b->kv_lens) || !aligned4(b->cu_rows))
    return bad(who, "page_table, kv_lens and cu_rows must be 4-byte aligned");
  if (b->table_stride < b->pages_per_seq) return bad(who, "table_stride must be at least pages_per_seq");
  if ((int64_t)b->pages_per_seq * c->page_tokens > (1 << 30)) return bad(who, "more than 2^30 positions a sequence");
  if (!b->cu_rows && b->rows % b->batch != 0) return bad(who, "without cu_rows rows must be a multiple of batch");
  if (!b->cu_rows && b->rows / b->batch > b->max_new) return bad(who, "max_new is smaller than rows / batch");
  a->codes = (uint8_t*)c->codes;
  a->scales = c->scales;
  a->table = b->page_table;
  a->table_stride = b->table_stride;
  a->lens = b->kv_lens;
  a->cu = b->cu_rows;
  a->per_seq = b->cu_rows ? 0 : b->rows / b->batch;
  a->B = b->batch;
  a->T = b->rows;
  a->max_new = b->cu_rows ? (b->max_new < b->rows ? b->max_new : b->rows) : a->per_seq;
  a->n_pages = c->n_pages;
  a->max_len = b->pages_per_seq * c->page_tokens;
  a->Hk = c->kv_heads;
  a->D = c->head_dim;
  a->lb = log2i(c->page_tokens / 16);
  if ((int64_t)a->B * (a->max_new / 16 + 2) > kMaxGrid) return bad(who, "batch * max_new is too large");
  return MOE_OK;
}

// (the kernels' factor of scores is scale * log2(e))
bool scale_ok(float scale) { return scale > 0 && isfinite(scale * kLog2e); }

int check_heads(const char* who, int q_heads, int kv_heads) {
  if (q_heads < 1 || q_heads > 4096 || q_heads % kv_heads != 0)
    return bad(who, "q_heads must be a multiple of kv_heads, at most 4096");
  return MOE_OK;
}

// Grids of the attention kernels: 16-row tiles in the third dimension, a join for each row.
int check_attn_grid(const char* who, int64_t batch, int64_t max_new, int64_t max_len, int64_t q_heads, int64_t kv_heads) {
  if ((max_new * (q_heads / kv_heads) + 15) / 16 > 65535 || batch * max_new > kMaxGrid)
    return bad(who, "batch, max_new or heads too large");
  // the kernels number the steps of 32 positions of all sequences in 32 bits
  if (batch * ((max_len + 31) / 32) > 0x7FFFFFFF - (1 << 20)) return bad(who, "batch * pages_per_seq * page_tokens too large");
  return MOE_OK;
}

struct AttnWs {
  size_t o, ml, where, total;
};

// `n` ranges over B contexts make at most n + B - 1 parts.
AttnWs attn_ws(int n, const KvArgs& kv, int q_heads) {
  AttnWs w{0, 0, 0, kAlign};
  if (n > 1) {
    const size_t rows = ((size_t)n + kv.B) * kv.max_new * q_heads;
    w.ml = align_up(rows * kv.D * 4);
    w.where = w.ml + align_up(rows * 8);
    w.total = w.where + align_up((size_t)kv.B * 8);
  }
  return w;
}

}  // namespace

extern "C" size_t moe_kv_code_bytes(int32_t n_pages, int32_t page_tokens, int32_t kv_heads, int32_t head_dim) {
  if (!geometry_ok(n_pages, page_tokens, kv_heads) || !dim_ok(head_dim)) return 0;
  return (size_t)n_pages * kv_heads * page_tokens * 2 * head_dim;
}

extern "C" size_t moe_kv_scale_bytes(int32_t n_pages, int32_t page_tokens, int32_t kv_heads) {
  if (!geometry_ok(n_pages, page_tokens, kv_heads)) return 0;
  return (size_t)n_pages * kv_heads * (page_tokens / 16) * 2 * 4;
}

extern "C" int moe_rope_freqs(int32_t rot_dim, double base, int rule, double factor, double trained, double slow,
                              double fast, double* freqs_out) {
  clear_error();
  static const char* who = "moe_rope_freqs";
  if (!freqs_out) return bad(who, "freqs_out is NULL");
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0) return bad(who, "rot_dim must be a multiple of 16 in [16, 256]");
  if (!(base > 1) || !isfinite(base)) return bad(who, "base must be finite and larger than 1");
  if (rule < MOE_ROPE_PLAIN || rule > MOE_ROPE_PARTS) return bad(who, "unknown rule");
  if (rule != MOE_ROPE_PLAIN && (!(factor >= 1) || !isfinite(factor))) return bad(who, "factor must be finite and at least 1");
  if (rule == MOE_ROPE_PARTS &&
      (!(trained > 0) || !(slow >= 0) || !(fast > slow) || !isfinite(trained) || !isfinite(fast)))
    return bad(who, "need trained > 0 and 0 <= slow < fast, finite");
  if (rule == MOE_ROPE_BASE) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
  if (!isfinite(base)) return bad(who, "base must be finite");
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (rule == MOE_ROPE_LINEAR) f /= factor;
    if (rule == MOE_ROPE_PARTS) {
      const double r = trained * f / 6.283185307179586;
      const double u = r >= fast ? 1.0 : r <= slow ? 0.0 : (r - slow) / (fast - slow);
      f = (1.0 - u) * (f / factor) + u * f;
    }
    freqs_out[i] = f;
  }
  return MOE_OK;
}

extern "C" int moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_rope* rope, int dtype,
                             const void* q, int64_t q_stride, int32_t q_heads, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride, void* k_out,
                             int64_t k_out_stride, void* stream) {
  clear_error();
  static const char* who = "moe_kv_append";
  AppendArgs a{};
  int rc = check_cache(who, cache, batch, &a.kv);
  if (rc != MOE_OK) return rc;
  if ((rc = check_dtype(who, dtype)) != MOE_OK) return rc;
  const int D = a.kv.D, Hk = a.kv.Hk;
  if ((rc = check_rows(who, "k", k, k_stride, Hk, D)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "v", v, v_stride, Hk, D)) != MOE_OK) return rc;
  if (k_out && (rc = check_rows(who, "k_out", k_out, k_out_stride, Hk, D)) != MOE_OK) return rc;
  if (q || q_out || q_heads) {
    if (q_heads < 1 || q_heads > 4096) return bad(who, "q_heads must be in [1, 4096] (0 without q)");
    if ((rc = check_rows(who, "q", q, q_stride, q_heads, D)) != MOE_OK) return rc;
    if ((rc = check_rows(who, "q_out", q_out, q_out_stride, q_heads, D)) != MOE_OK) return rc;
    a.Hq = q_heads;
  }
  // (in place means the very same rows: another stride or start would let a
  // head's output reach rows that are still to be read)
  if (q && q_out == q && q_out_stride != q_stride) return bad(who, "q_out in place of q needs q's stride");
  if (k_out == k && k_out_stride != k_stride) return bad(who, "k_out in place of k needs k's stride");
  if (rope && rope->rot_dim != 0) {
    if (rope->rot_dim < 16 || rope->rot_dim % 16 != 0 || rope->rot_dim > D)
      return bad(who, "rot_dim must be 0 or a multiple of 16, at most head_dim");
    if (!rope->freqs) return bad(who, "rope has no frequencies");
    if (((uintptr_t)rope->freqs & 7u) != 0) return bad(who, "rope's frequencies must be 8-byte aligned");
    if (!isfinite(rope->scale)) return bad(who, "rope's scale must be finite");
    a.rot = rope->rot_dim;
    a.inter = rope->interleaved != 0;
    a.rscale = rope->scale;
    a.freqs = rope->freqs;
  }
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_out = k_out;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  hipError_t e = launch_kv_append(a, dtype, n_cus(), (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : hip_fail(who, e);
}

extern "C" int moe_kv_read(const moe_kv_cache* cache, const moe_kv_batch* batch, int dtype, void* k_out,
                           int64_t k_out_stride, void* v_out, int64_t v_out_stride, void* stream) {
  clear_error();
  static const char* who = "moe_kv_read";
  ReadArgs a{};
  int rc = check_cache(who, cache, batch, &a.kv);
  if (rc != MOE_OK) return rc;
  if ((rc = check_dtype(who, dtype)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "k_out", k_out, k_out_stride, a.kv.Hk, a.kv.D)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "v_out", v_out, v_out_stride, a.kv.Hk, a.kv.D)) != MOE_OK) return rc;
  a.k_out = k_out;
  a.v_out = v_out;
  a.kos = k_out_stride;
  a.vos = v_out_stride;
  hipError_t e = launch_kv_read(a, dtype, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : hip_fail(who, e);
}

namespace {

int check_decode_args(const char* who, const moe_kv_cache* cache, const moe_kv_batch* batch, int32_t q_heads, KvArgs* kv) {
  int rc = check_cache(who, cache, batch, kv);
  if (rc != MOE_OK) return rc;
  if ((rc = check_heads(who, q_heads, kv->Hk)) != MOE_OK) return rc;
  return check_attn_grid(who, kv->B, kv->max_new, kv->max_len, q_heads, kv->Hk);
}

}  // namespace

extern "C" size_t moe_attn_decode_workspace_bytes(const moe_kv_cache* cache, const moe_kv_batch* batch,
                                                  int32_t q_heads) {
  clear_error();
  KvArgs kv{};
  if (check_decode_args("moe_attn_decode_workspace_bytes", cache, batch, q_heads, &kv) != MOE_OK) return 0;
  return attn_ws(attn_decode_workers(kv, q_heads, n_cus()), kv, q_heads).total;
}

extern "C" int moe_attn_decode(const moe_kv_cache* cache, const moe_kv_batch* batch, int dtype, const void* q,
                               int64_t q_stride, int32_t q_heads, float scale, void* out, int64_t out_stride,
                               float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  static const char* who = "moe_attn_decode";
  DecodeArgs a{};
  int rc = check_decode_args(who, cache, batch, q_heads, &a.kv);
  if (rc != MOE_OK) return rc;
  if ((rc = check_dtype(who, dtype)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "q", q, q_stride, q_heads, a.kv.D)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "out", out, out_stride, q_heads, a.kv.D)) != MOE_OK) return rc;
  if (!scale_ok(scale)) return bad(who, "scale must be positive, and finite times log2(e)");
  if (!aligned4(lse)) return bad(who, "lse must be 4-byte aligned");
  if (!ws || !aligned16(ws)) return bad(who, "ws must be 16-byte aligned memory");
  const int n = attn_decode_workers(a.kv, q_heads, n_cus());
  const AttnWs w = attn_ws(n, a.kv, q_heads);
  if (ws_bytes < w.total)
    return fail(MOE_ERR_WORKSPACE, std::string(who) + ": workspace too small (need " + std::to_string(w.total) + ")");
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.qs = q_stride;
  a.os = out_stride;
  a.Hq = q_heads;
  a.c = scale * kLog2e;
  a.split = {(float*)((uint8_t*)ws + w.o), (float*)((uint8_t*)ws + w.ml), (int2*)((uint8_t*)ws + w.where), n};
  hipError_t e = launch_attn_decode(a, dtype, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : hip_fail(who, e);
}

namespace {

int check_packed(const char* who, const moe_packed* p, PrefillArgs* a) {
  if (!p) return bad(who, "the packed description is NULL");
  if (p->batch < 1 || p->batch > kMaxBatch || p->rows_q < 1 || p->rows_q > kMaxRows || p->rows_k < 0 || p->rows_k > kMaxRows || p->max_q < 1)
    return bad(who, "need batch, rows_q and max_q >= 1, rows_k >= 0, batch <= 2^20, rows <= 2^24");
  if (p->kv_heads < 1 || p->kv_heads > 256) return bad(who, "need 1 <= kv_heads <= 256");
  int rc = check_heads(who, p->q_heads, p->kv_heads);
  if (rc != MOE_OK) return rc;
  if (!dim_ok(p->head_dim)) return fail(MOE_ERR_UNSUPPORTED, std::string(who) + ": head_dim must be 64, 128 or 256");
  if (!aligned4(p->cu_q) || !aligned4(p->cu_k)) return bad(who, "cu_q and cu_k must be 4-byte aligned");
  if (!p->cu_q && p->rows_q % p->batch != 0) return bad(who, "without cu_q rows_q must be a multiple of batch");
  if (!p->cu_k && p->rows_k % p->batch != 0) return bad(who, "without cu_k rows_k must be a multiple of batch");
  if (!p->cu_q && p->rows_q / p->batch > p->max_q) return bad(who, "max_q is smaller than rows_q / batch");
  a->cu_q = p->cu_q;
  a->cu_k = p->cu_k;
  a->B = p->batch;
  a->Tq = p->rows_q;
  a->Tk = p->rows_k;
  a->per_q = p->cu_q ? 0 : p->rows_q / p->batch;
  a->per_k = p->cu_k ? 0 : p->rows_k / p->batch;
  a->max_q = p->cu_q ? (p->max_q < p->rows_q ? p->max_q : p->rows_q) : a->per_q;
  a->Hq = p->q_heads;
  a->Hk = p->kv_heads;
  a->D = p->head_dim;
  // (row tiles of 128, whole rounds of 8 XCDs)
  if ((int64_t)a->max_q * (a->Hq / a->Hk) > (1 << 30) ||
      ((((int64_t)a->max_q * (a->Hq / a->Hk) + 127) / 128) * a->Hk + 7) * a->B > kMaxGrid)
    return bad(who, "batch, max_q or heads too large");
  return MOE_OK;
}

AttnWs prefill_ws(const PrefillArgs& a, int n) {
  AttnWs w{0, 0, 0, kAlign};
  if (n > 1) {
    const size_t rows = (size_t)n * a.Tq * a.Hq;
    w.ml = align_up(rows * a.D * 4);
    w.total = w.ml + align_up(rows * 8);
  }
  return w;
}

}  // namespace

extern "C" size_t moe_attn_prefill_workspace_bytes(const moe_packed* p) {
  clear_error();
  PrefillArgs a{};
  if (check_packed("moe_attn_prefill_workspace_bytes", p, &a) != MOE_OK) return 0;
  return prefill_ws(a, attn_prefill_parts(a, n_cus())).total;
}

extern "C" int moe_attn_prefill(const moe_packed* p, int dtype, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, float scale, int causal, void* out,
                                int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  static const char* who = "moe_attn_prefill";
  PrefillArgs a{};
  int rc = check_packed(who, p, &a);
  if (rc != MOE_OK) return rc;
  if ((rc = check_dtype(who, dtype)) != MOE_OK) return rc;
  if ((rc = check_rows(who, "q", q, q_stride, a.Hq, a.D)) != MOE_OK) return rc;
  if (a.Tk > 0) {
    if ((rc = check_rows(who, "k", k, k_stride, a.Hk, a.D)) != MOE_OK) return rc;
    if ((rc = check_rows(who, "v", v, v_stride, a.Hk, a.D)) != MOE_OK) return rc;
  }
  if ((rc = check_rows(who, "out", out, out_stride, a.Hq, a.D)) != MOE_OK) return rc;
  if (!scale_ok(scale)) return bad(who, "scale must be positive, and finite times log2(e)");
  if (!aligned4(lse)) return bad(who, "lse must be 4-byte aligned");
  if (!ws || !aligned16(ws)) return bad(who, "ws must be 16-byte aligned memory");
  const int n = attn_prefill_parts(a, n_cus());
  const AttnWs w = prefill_ws(a, n);
  if (ws_bytes < w.total)
    return fail(MOE_ERR_WORKSPACE, std::string(who) + ": workspace too small (need " + std::to_string(w.total) + ")");
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.os = out_stride;
  a.c = scale * kLog2e;
  a.causal = causal != 0;
  a.split = {(float*)((uint8_t*)ws + w.o), (float*)((uint8_t*)ws + w.ml), nullptr, n};
  hipError_t e = launch_attn_prefill(a, dtype, (hipStream_t)stream);
  return e == hipSuccess ? MOE_OK : hip_fail(who, e);
}

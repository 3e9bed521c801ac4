// Launch interface of the attention kernels (k_kv.hip, k_attn_decode.hip,
// k_attn_prefill.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmoe {

// A cache and a step's sequences over it (include/qmoe_attn.h).
struct KvArgs {
  uint8_t* codes;
  float* scales;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu;        // null: per_seq rows each
  int per_seq;
  int B, T, max_new;
  int n_pages, max_len;     // max_len = pages_per_seq * page_tokens
  int Hk, D;
  int lb;                   // log2 of the blocks of a page
};

struct AppendArgs {
  KvArgs kv;
  const void *q, *k, *v;
  void *q_out, *k_out;
  int64_t qs, ks, vs, qos, kos;
  int Hq;                   // 0: no q
  int rot, inter;
  float rscale;
  const double* freqs;
};
hipError_t launch_kv_append(const AppendArgs& a, int dtype, int cus, hipStream_t s);

struct ReadArgs {
  KvArgs kv;
  void *k_out, *v_out;
  int64_t kos, vos;
};
hipError_t launch_kv_read(const ReadArgs& a, int dtype, hipStream_t s);

// Sums of parts of contexts, for the join: un-normalised outputs
// [part][max_new][Hq][D] and (maximum in powers of two, sum)
// [part][max_new][Hq][2], and for each sequence its first part's range and
// its number of parts.
struct SplitBuf {
  float* o;
  float* ml;
  int2* where;
  int n;                    // ranges the contexts are cut into (1: no join)
};

struct DecodeArgs {
  KvArgs kv;
  const void* q;
  void* out;
  float* lse;
  int64_t qs, os;
  int Hq;
  float c;                  // scale * log2(e)
  SplitBuf split;
};
int attn_decode_workers(const KvArgs& kv, int Hq, int cus);
hipError_t launch_attn_decode(const DecodeArgs& a, int dtype, hipStream_t s);

struct PrefillArgs {
  const int32_t *cu_q, *cu_k;
  int B, Tq, Tk, max_q, per_q, per_k;
  int Hq, Hk, D;
  const void *q, *k, *v;
  void* out;
  float* lse;
  int64_t qs, ks, vs, os;
  float c;
  int causal;
  SplitBuf split;           // parts [part][Tq][Hq] of the keys (where: unused)
};
int attn_prefill_parts(const PrefillArgs& a, int cus);
hipError_t launch_attn_prefill(const PrefillArgs& a, int dtype, hipStream_t s);

}  // namespace qmoe

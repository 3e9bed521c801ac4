/*
 * qmoe_step.h -- C ABI of the calls of libqmoe that stand around the routed
 * experts (include/qmoe.h) and attention (include/qmoe_attn.h) in a serving
 * step on AMD Instinct MI355X (gfx950): the residual's addition and the
 * root-mean-square norm, products of a few rows with 4-bit weights (the
 * projections around attention, the logits), and the keeping of a paged
 * cache's pages on the GPU.  Conventions are those of the other two headers:
 * the caller owns every buffer, device base pointers are 16-byte aligned
 * memory of the current device (arrays of int32 4-byte aligned), calls
 * enqueue kernels on `stream` and return without waiting, arguments are
 * checked on the host before anything is enqueued, a failing call returns a
 * MOE_ERR_* code, touches no output and leaves a message for moe_last_error();
 * results do not depend on the order in which the GPU works (integer counts
 * are the only atomics).  Every call may be captured into a HIP graph.
 */
#ifndef QMOE_STEP_H
#define QMOE_STEP_H

#include "qmoe_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DT_F32 2
#define MOE_DT_I8 3

/* ---------------------------------------------------------------------------
 * Norm.
 *
 * Rows of `heads` vectors of `cols` values, a row's vectors back to back, rows
 * `stride` elements apart (a multiple of 8, at least heads * cols, at most
 * 2^24).  Every vector is normed by itself (heads = 1: the hidden rows of a
 * layer; more: queries' or keys' heads).  cols is a multiple of 8, 8 to 16384;
 * heads is 1 to 4096; rows * heads is below 2^24, where cols > 2048 below 2^23,
 * where cols > 4096 below 2^22.
 * Types: MOE_DT_BF16, MOE_DT_F16, MOE_DT_F32.
 *
 *   h = x + residual, added in 32 bits and rounded to the residual's type
 *       (without a residual: x), which `sum` gets where it is not NULL;
 *   y = h * weight / sqrt(mean(h^2) + eps)   (weight NULL: 1)
 *
 * out: y rounded to out_dtype; NULL: not wanted.
 * codes, scales: y in 8 bits; NULL both: not wanted.  Columns share a scale
 *   in groups of `group` (128, the last perhaps shorter; 0: the whole vector):
 *     m = max |y| rounded to 32 bits,  scale = m / 127 rounded to 32 bits,
 *     code = y / scale rounded to the nearest integer (ties to even), at most
 *     127 in size, 0 where scale is 0;
 *   y here is not out's rounded one: it is taken in 64 bits, so that codes
 *   next to a border fall as in exact arithmetic.  Where m is infinite or not
 *   a number the scale is not a number and the codes are 0.
 *   codes int8 as the rows of out, codes_stride apart; the scale of row r,
 *   vector v, group g is scales[(v * groups + g) * scale_stride + r], with
 *   scale_stride a multiple of 4, at least rows, at most 2^28.
 * Sums of squares are 64-bit (no overflow for any input).
 * At least one of out, codes and sum is wanted; sum needs a residual.  sum may
 * be x or the residual, and out too, where type and stride are the same, so
 * that each row takes its own place; outputs must not overlap inputs or each
 * other otherwise.  rows = 0: nothing is done (the rows may be NULL). */
typedef struct moe_norm {
  int32_t rows;
  int32_t heads;
  int32_t cols;
  int32_t x_dtype;
  const void* x;
  int64_t x_stride;
  int32_t residual_dtype;
  int32_t weight_dtype;
  const void* residual;
  int64_t residual_stride;
  void* sum;
  int64_t sum_stride;
  const void* weight;
  float eps;
  int32_t out_dtype;
  void* out;
  int64_t out_stride;
  int8_t* codes;
  int64_t codes_stride;
  float* scales;
  int64_t scale_stride;
  int32_t group;
} moe_norm;

int moe_rms_norm(const moe_norm* norm, void* stream);

/* ---------------------------------------------------------------------------
 * Products with 4-bit weights.
 *
 * A matrix [n, k] of codes q = 0..15; groups of `group` (32, 64 or 128)
 * consecutive columns of a row share an fp16 scale s and a zero point z = 0..15
 * (8 everywhere for a matrix without zero points): weight = s (q - z).  The
 * last group of a row may be shorter.  k is a multiple of 8, 8 to 2^20; n is 1 to
 * 2^24.
 *
 * Packed: tiles of 16 rows x 128 columns, tile (rt, kc) (rt = row / 16,
 * kc = column / 128) at (rt * ceil(k/128) + kc) * TILE, with codes of 8, scales of 0 and
 * zero points of 8 where a tile reaches past the matrix, and gt = 128 / group:
 *   [0, 1024)          lane c = 16*g + r at 16*c holds 4 words; word i has the
 *                      codes of row r, columns 32*i + 8*g + j: that of j = 0..7
 *                      at bit 4*(j/2) + 16*(j%2), stored as q ^ 8
 *   [1024, +32*gt)     row r at 2*gt*r: the scales of its groups
 *   then, with zero points, [.., +16*gt): row r at gt*r: bytes z - 8
 */

/* Host only.  Codes (uint8 [n][k]), scales (fp16 bits [n][ceil(k/group)]) and,
 * where zeros is not NULL, zero points (uint8 [n][ceil(k/group)]) of an fp32
 * host matrix [n][k], by rounding to nearest in 64 bits:
 *   without zero points  s = fp16(max |w| / 7), z = 8,
 *                        q = clamp(floor(w/s + 1/2) + 8, 0, 15)
 *   with                 lo = min(0, min w), hi = max(0, max w),
 *                        s = fp16((hi - lo) / 15), z = clamp(floor(-lo/s + 1/2), 0, 15),
 *                        q = clamp(floor(w/s + 1/2) + z, 0, 15)
 * (s = 0: q = z = 8).  MOE_ERR_INVALID_ARG for a bad shape, NULL, a value that
 * is not finite, or a scale that fp16 does not hold; nothing is written then. */
int moe_linear_quantize(const float* w, int64_t n, int64_t k, int32_t group, uint8_t* codes, uint16_t* scales,
                        uint8_t* zeros, int n_threads);

/* Host only.  Bytes of a packed matrix (0 for a bad shape), and the packing of
 * codes, scales and zero points (NULL: none) as above.  MOE_ERR_INVALID_ARG
 * for a bad shape, NULL, codes or zero points above 15, scales that are not finite, or
 * out_bytes too small; nothing is written then.  n_threads 0: the machine's. */
size_t moe_linear_packed_bytes(int64_t n, int64_t k, int32_t group, int with_zeros);
int moe_linear_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t n, int64_t k,
                    int32_t group, void* out, size_t out_bytes, int n_threads);

/* A packed matrix in device memory; bias: device float [n] or NULL. */
typedef struct moe_linear_weights {
  int32_t n;
  int32_t k;
  int32_t group;
  int32_t with_zeros;
  const void* packed;
  const float* bias;
} moe_linear_weights;

/* y[t, i] = sum_j x[t, j] weight[i, j] + bias[i] for rows t = 0..rows-1.
 *   x     x_dtype MOE_DT_BF16, MOE_DT_F16, or MOE_DT_I8: codes (-128..127) with
 *         scales, value = code * scale.  Rows x_stride elements apart (a
 *         multiple of 8, at least k, at most 2^24).
 *   x_scales  (MOE_DT_I8; NULL otherwise) as moe_rms_norm writes them for one
 *         vector a row: that of row t, group g at x_scales[g * scale_stride + t]
 *         (scale_stride a multiple of 4, at least rows, at most 2^28);
 *         x_group 128, or 0: one scale a row.  The last group too has scale_stride
 *         of them, read up to the next multiple of 4 rows.
 *   y     y_dtype MOE_DT_BF16, MOE_DT_F16 or MOE_DT_F32, rows y_stride elements apart (at
 *         least n, at most 2^24).
 * Codes and products are exact; 16-bit rows' sums are 32-bit ones, 8-bit
 * rows' are exact inside a group of columns that share both scales and 32-bit
 * between them; the result is rounded once.  16-bit rows: a group's sum is
 * 16 s (sum x (1 + q/16) - (1 + z/16) sum x), so that y is off by up to
 * 2^-23 * 64 * (group + 4) * sum |x_j s_j| (measured: 2^-20 of sum |x_j s_j|
 * for k = 128, 2^-24 for k = 4096), and weights at their zero points can give
 * something of that size, not 0.  16-bit rows: twice the sum of a
 * group's |x| must be below 2^128, or the row overflows.  A row that holds a
 * value that is not finite gives infinities or not a number; other rows are
 * not touched by it.  Meant for few rows (the weights are read from memory
 * once for each 64); any number up to 2^20 works.  rows = 0: nothing is done
 * (the rows may be NULL).  y must not overlap the inputs. */
int moe_linear(const moe_linear_weights* w, int32_t rows, int x_dtype, const void* x, int64_t x_stride,
               const float* x_scales, int64_t scale_stride, int32_t x_group, int y_dtype, void* y, int64_t y_stride,
               void* stream);

/* ---------------------------------------------------------------------------
 * Pages of a cache (include/qmoe_attn.h), kept on the GPU.
 *
 * A pool: n_pages (1 to 2^29) pages, which every one of its caches holds a part
 * of, and refs, device int32 [n_pages]: how many table entries name each page,
 * 0: free.  A new pool is refs of zeros.  caches is a host array of n_caches (0
 * to 256: a model's layers), read during the call; they may differ in heads, not
 * in n_pages and page_tokens, and their scales may be 4-byte aligned here.
 * Calls on one pool, or on one page table, must come one after the other (one
 * stream, or events between). */
typedef struct moe_kv_pool {
  int32_t n_pages;
  int32_t n_caches;
  const moe_kv_cache* caches;
  int32_t* refs;
} moe_kv_pool;

/* Rows of a page table, one a sequence: row b, of kv_lens[b] positions, holds
 * pages page_table[b][0 .. held-1], held = ceil(kv_lens[b] / page_tokens).
 * page_table: device int32 [seqs][pages_per_seq], rows table_stride apart;
 * kv_lens: device int32 [seqs].  These are moe_kv_batch's.  seqs is 1 to 4096,
 * seqs * pages_per_seq at most 2^30, pages_per_seq * page_tokens too.
 * Lengths outside [0, pages_per_seq * page_tokens] count as the nearest in it;
 * an entry that names no page of the pool is passed over. */
typedef struct moe_kv_tables {
  int32_t seqs;
  int32_t pages_per_seq;
  int32_t page_tokens;
  int32_t* page_table;
  int64_t table_stride;
  int32_t* kv_lens;
} moe_kv_tables;

/* Gives every row b the length new_lens[b] (device int32 [seqs]; negative: the
 * row is left alone).  First rows that get shorter give back the pages they no
 * longer need (their entries become -1; a page is free when its last holder
 * gives it back).
 * Then rows that get longer take free pages: the lowest ids, in ascending order
 * of row and position.  When there are too few, the rows up to the first
 * one that lacks pages get theirs, and that one and the later ones that
 * need any stay as they are.  missing (device int32 [1], NULL: not wanted): the
 * pages that rows needed and did not get.
 * A row that is cut back into a page which others hold must be forked from itself
 * (below) before it is appended to.  new_lens must not be kv_lens. */
int moe_kv_resize(const moe_kv_pool* pool, const moe_kv_tables* tables, const int32_t* new_lens, int32_t* missing,
                  void* stream);

/* Lets row b go on from row a = from[b] (device int32 [seqs]; outside of [0,
 * seqs): row b is left alone).  Row b has to be of length 0 and row a longer
 * (both before the call; other rows b are left alone).  Row b gets row a's
 * length, shares its full pages, and gets a page of its own for the positions
 * behind them, whose blocks of 16 positions are copied in every cache.
 * from[b] = b: where row b ends inside a page that others hold too, it gets a
 * copy of that page of its own instead.
 * Pages are taken and `missing` counted as by moe_kv_resize (a row that lacks
 * its page stays as it is); pages that this call frees are not taken in it.
 * ws: device scratch, no initialization needed; calls that overlap in
 * time need one each. */
size_t moe_kv_fork_workspace_bytes(const moe_kv_pool* pool, const moe_kv_tables* tables);
int moe_kv_fork(const moe_kv_pool* pool, const moe_kv_tables* tables, const int32_t* from, int32_t* missing, void* ws,
                size_t ws_bytes, void* stream);

/* Moves held pages (refs not 0) to the low end of the pool: with n of them,
 * those with ids from n on, in ascending order, go into the free ids below n, in
 * ascending order; the caches' pages, refs and the rows' entries follow.
 * Entries that name a moved page must all be among the rows of `tables`.
 * held (device int32 [1], NULL: not wanted): n.  ws as for moe_kv_fork. */
size_t moe_kv_compact_workspace_bytes(const moe_kv_pool* pool, const moe_kv_tables* tables);
int moe_kv_compact(const moe_kv_pool* pool, const moe_kv_tables* tables, int32_t* held, void* ws, size_t ws_bytes,
                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMOE_STEP_H */

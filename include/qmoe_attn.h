/*
 * qmoe_attn.h -- C ABI of the attention calls of libqmoe for AMD Instinct
 * MI355X (gfx950): rotary positions, a paged key/value cache held in 8 bits,
 * attention of a few new tokens over that cache, and attention of packed
 * prompts.  They are the attention half of the layer step whose expert half
 * include/qmoe.h declares, with its conventions: the caller owns every
 * buffer, device base pointers are 16-byte aligned memory of the current
 * device, calls enqueue kernels on `stream` and return without waiting,
 * arguments are checked on the host before anything is enqueued, a failing
 * call returns a MOE_ERR_* code, touches no output and leaves a message for
 * moe_last_error(); results are fixed-order computations (no atomics).
 * Every call may be captured into a HIP graph.
 *
 * What lies in device memory (page tables, lengths, row offsets) cannot be
 * checked on the host; the kernels clamp it, so that no value there makes
 * them touch memory outside the buffers the arguments describe:
 *   lengths to [0, pages_per_seq * page_tokens], row offsets to [0, rows]
 *   in ascending order; a page id outside [0, n_pages) is a page of no
 *   tokens (nothing is written to it, it reads as zeros, attention leaves
 *   its tokens out).
 *
 * Row tensors (q, k, v, outputs): [rows][heads][head_dim] of one 16-bit type
 * (MOE_DT_BF16 or MOE_DT_F16), a row's heads back to back, rows `stride`
 * elements apart (a multiple of 8, at least heads * head_dim, at most 2^24), so
 * q, k and v may be parts of one projection's output.  head_dim is 64, 128 or 256;
 * q_heads is a multiple of kv_heads, query head h reads key head
 * h / (q_heads / kv_heads).
 */
#ifndef QMOE_ATTN_H
#define QMOE_ATTN_H

#include "qmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DT_BF16 0
#define MOE_DT_F16 1

/* The cache.  A page holds page_tokens positions of one sequence (a power of
 * two, 16 to 1024) of every key head; a block is 16 of them (aligned) of one
 * head.
 *
 * codes: uint8 [n_pages][kv_heads][page_tokens/16][2][16*head_dim], K codes
 *   of the block and then V codes; values are 8-bit floating-point numbers
 *   with 4 exponent and 3 mantissa bits (bias 7, largest 448, 0x7F and 0xFF
 *   not a number).  With lane c = 16*g + n (g = 0..3, n = 0..15):
 *     K: piece h = 0..head_dim/64-1 at 1024*h: lane c at 16*c holds, of token
 *        n, columns 64*h + 8*g + (0..7), then 64*h + 32 + 8*g + (0..7).
 *     V: piece h at 1024*h: lane c at 16*c holds words w = 0..3 of column
 *        64*h + 16*w + n: byte i is token 4*g + i.
 *   So one 16-byte load per lane is the matrix core's operand.
 * scales: float [n_pages][kv_heads][page_tokens/16][2]: the scales of the
 *   block's K and V; value = code * scale.  moe_kv_append writes powers of
 *   two from 2^-64 to 2^121, whatever else fills a cache keeps to that range, and
 *   the readers use the exponent only.
 */
typedef struct moe_kv_cache {
  int32_t n_pages;
  int32_t page_tokens;
  int32_t kv_heads;
  int32_t head_dim;
  void* codes;
  float* scales;
} moe_kv_cache;

/* Bytes of `codes` and of `scales` (0 for a bad geometry). */
size_t moe_kv_code_bytes(int32_t n_pages, int32_t page_tokens, int32_t kv_heads, int32_t head_dim);
size_t moe_kv_scale_bytes(int32_t n_pages, int32_t page_tokens, int32_t kv_heads);

/* A step of `batch` sequences with `rows` rows in all.
 *   page_table  device int32 [batch][pages_per_seq], rows table_stride
 *               apart: page p of sequence b holds its positions
 *               p*page_tokens to (p+1)*page_tokens - 1.
 *   kv_lens     device int32 [batch]: positions each sequence has, those of
 *               this step's rows included.
 *   cu_rows     device int32 [batch+1]: sequence b has rows cu_rows[b] to
 *               cu_rows[b+1]-1; NULL: rows/batch each.
 *   max_new     at least the largest number of rows of one sequence
 *               (attention leaves rows past it as they are, appending and
 *               reading may).
 * Row i of the n rows of sequence b is position kv_lens[b] - n + i: the
 * step's rows are the sequence's last.  Rows behind cu_rows[batch] are left
 * as they are. */
typedef struct moe_kv_batch {
  int32_t batch;
  int32_t rows;
  int32_t max_new;
  int32_t pages_per_seq;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* kv_lens;
  const int32_t* cu_rows;
} moe_kv_batch;

/* Rotary positions: the first rot_dim columns of a head (a multiple of 16,
 * at most head_dim) are turned in pairs i = 0..rot_dim/2-1, columns
 * (i, i + rot_dim/2) or with `interleaved` (2i, 2i+1):
 *   a' = scale (a cos t - b sin t), b' = scale (a sin t + b cos t),
 *   t = position * freqs[i].
 * freqs: device double [rot_dim/2], radians a position.  t is reduced in 64
 * bits, so far positions keep their angle. */
typedef struct moe_rope {
  int32_t rot_dim;
  int32_t interleaved;
  float scale;
  const double* freqs;
} moe_rope;

#define MOE_ROPE_PLAIN 0
#define MOE_ROPE_LINEAR 1
#define MOE_ROPE_BASE 2
#define MOE_ROPE_PARTS 3

/* Host only.  The table of frequencies (host double [rot_dim/2]) for
 * contexts `factor` times as long as the trained one:
 *   PLAIN   f_i = base^(-2i/rot_dim)
 *   LINEAR  f_i / factor
 *   BASE    base * factor^(rot_dim/(rot_dim-2)) in place of base (the slowest
 *           pair is slowed by factor, the fastest not at all)
 *   PARTS   by the turns r = trained * f_i / (2 pi) a pair makes over the
 *           trained length: f_i for r >= fast, f_i / factor for r <= slow,
 *           between them (1-u) f_i/factor + u f_i, u = (r-slow)/(fast-slow).
 * (Scaling rules: Chen et al. 2023, "Extending Context Window of Large
 * Language Models via Positional Interpolation"; Peng et al. 2023, "YaRN".)
 * MOE_ERR_INVALID_ARG for rot_dim not a positive multiple of 16 (<= 256),
 * base <= 1, factor < 1 (but for PLAIN, which has none), PARTS without 0 <= slow < fast and trained > 0, BASE
 * with rot_dim < 4, numbers not finite, an unknown rule or NULL. */
int moe_rope_freqs(int32_t rot_dim, double base, int rule, double factor, double trained, double slow,
                   double fast, double* freqs_out);

/* Turns the step's q and k rows by their positions and appends the k and v
 * rows to the cache.
 *   rope    NULL (or rot_dim 0): no turn.
 *   q       turned into q_out (which may be q itself); NULL with q_heads 0:
 *           no q.
 *   k_out   the turned k rows, rounded once to the row type (may be k
 *           itself); NULL: not wanted.
 * q is turned in 32 bits; k in 64, with sines and cosines good to 2^-40, and
 * k_out and the codes are the turned values rounded once (nearest, ties to
 * even).  Scale of a block's K (or V): the least power of two s, not below 2^-64,
 * with |x| <= 448 s for every finite x that was appended to the block since its
 * first slot was last written.  Tokens that were cut off again (a rejected
 * draft: kv_lens goes back, and the next step overwrites them) count among
 * those: the block keeps the scale they made it need, and its earlier tokens
 * the second rounding, until its first slot is written again.  (Where a
 * rejected draft must leave no trace, put the block's codes and scales back as
 * they were before it.)  A token that needs a larger scale than its block has
 * makes the earlier tokens' codes of that block be divided by the growth and
 * rounded again (exact but for values below 2^-6 of the new scale).
 * Infinities and NaN become the code for not a number.  The first slot of a
 * block starts a new scale, so pages may be reused without clearing.  Slots
 * behind the new tokens are left as they are.
 * Rows at negative positions (more rows than kv_lens) are turned but not
 * appended.  Two sequences of one step must not append to the same page
 * (they may share pages that neither appends to), nor one sequence to a page
 * that its table names twice.  q_out, k_out and the inputs must not overlap
 * otherwise. */
int moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_rope* rope, int dtype,
                  const void* q, int64_t q_stride, int32_t q_heads, const void* k, int64_t k_stride,
                  const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride, void* k_out,
                  int64_t k_out_stride, void* stream);

/* The step's positions out of the cache, as rows (with as many rows as a
 * sequence has positions, its whole context): code * scale, rounded to the
 * row type; beyond its range its largest number (65504 has code 256 at scale
 * 256).  Negative positions read as zeros.  Here rows need not be new
 * ones, only the sequence's last. */
int moe_kv_read(const moe_kv_cache* cache, const moe_kv_batch* batch, int dtype, void* k_out,
                int64_t k_out_stride, void* v_out, int64_t v_out_stride, void* stream);

/* Workspace bytes of moe_attn_decode (0 for invalid arguments; at least 256
 * otherwise).  It goes by batch, rows, max_new and pages_per_seq, not by what
 * device memory holds. */
size_t moe_attn_decode_workspace_bytes(const moe_kv_cache* cache, const moe_kv_batch* batch, int32_t q_heads);

/* Attention of each sequence's rows (its newest tokens, their own keys and
 * values already appended) over its cached positions:
 *   out[r,h] = sum_j p_j V_j, p = softmax_j(scale q[r,h] . K_j), over the
 *   positions j <= the row's own; a row with none of them gives zeros.
 * scale: positive, scale * log2(e) finite.
 * lse (device float [rows][q_heads], NULL: not wanted): log sum_j
 * exp(scale q . K_j), -inf for an empty row.  Codes and scales enter the
 * products exactly, whatever the row type's range is; a weight p is held to
 * 2^-16 of itself (a bf16 number and what its rounding leaves, as another);
 * sums are 32-bit, and the output is rounded once to the row type (a sum outside
 * its range gives infinity).  Meant for few rows a sequence
 * (1..16 in decoding and draft verification; any number works).  ws: device
 * scratch, no initialization needed; calls that overlap in time need one each.
 * out and lse must not overlap the inputs.
 * pages_per_seq * page_tokens, and not what kv_lens holds, chooses how contexts
 * are taken: up to 1024 positions (1536 where batch * kv_heads >= 32) by one
 * workgroup each, wider tables cut into ranges and joined by a second launch.
 * A program whose table has the width of its longest possible context may
 * describe the first pages of each row only (a smaller pages_per_seq with the
 * same table_stride) where they hold all the contexts of a step: one context of
 * 777 positions is then 7.6 us a call, 9.3 with a table of 32768. */
int moe_attn_decode(const moe_kv_cache* cache, const moe_kv_batch* batch, int dtype, const void* q,
                    int64_t q_stride, int32_t q_heads, float scale, void* out, int64_t out_stride, float* lse,
                    void* ws, size_t ws_bytes, void* stream);

/* Packed prompts: sequence b has query rows cu_q[b]..cu_q[b+1]-1 of rows_q
 * and key rows cu_k[b]..cu_k[b+1]-1 of rows_k (device int32 [batch+1];
 * NULL: rows/batch each).  max_q: at least the largest number of query rows
 * of one sequence (rows past it are left as they are). */
typedef struct moe_packed {
  int32_t batch;
  int32_t rows_q;
  int32_t rows_k;
  int32_t max_q;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
} moe_packed;

/* Workspace bytes of moe_attn_prefill (0 for invalid arguments; at least 256
 * otherwise). */
size_t moe_attn_prefill_workspace_bytes(const moe_packed* p);

/* Attention of packed sequences: as moe_attn_decode, with k and v rows in
 * place of the cache, and the weights p rounded to the row type: half a step
 * of each, fp16's below 2^-24 of the row's largest to a multiple of 2^-34 of it.
 * Scores are 32-bit sums, good to 2^-24 of the largest |score| among a row's
 * keys.  causal != 0: query row i of n sees key rows
 * j <= m - n + i of the sequence's m (aligned at the end: a chunk's rows come
 * last; with n > m the first n - m rows see nothing); else all m.  rows_k may
 * be 0 (k and v are not read then).  out, lse and ws as above. */
int moe_attn_prefill(const moe_packed* p, int dtype, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, float scale, int causal, void* out,
                     int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMOE_ATTN_H */

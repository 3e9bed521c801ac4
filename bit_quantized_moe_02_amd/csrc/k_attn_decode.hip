// Attention of a few new tokens of each sequence over its cached context
// (moe_attn_decode), and the join of parts of a context.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.hpp"

using namespace qmoe;
using namespace qmoe_dev;

namespace {

constexpr int kWaves = 4;                   // of a workgroup that takes a range
constexpr int kShortWaves = 8;              // of one that takes a whole short context
constexpr int kThreads = 256;               // of the join
constexpr int kStep = 32;                   // positions a wave takes at once: two blocks
constexpr float kLazy = 8.f;                // how far a score may exceed the running maximum, in powers of 2

// Shares.  The contexts of all sequences, in steps of 32 positions one after
// the other (a sequence with rows and no context counts as one step), are
// cut into `workers` equal ranges, so that every workgroup has the same work
// whatever the lengths are.  A worker's range is one or more segments, each
// of one sequence; a sequence that lies in one range needs no join.  The sums
// of worker w's segment of sequence b are part w + b: both only grow along
// the ranges, so no two segments share a number.
struct Cut {
  int per, total;                           // steps of a range, of all
};

// Inclusive sum over the lanes of a wave: within rows of 16 lanes, then the
// last lane of rows 0 and 2 to rows 1 and 3, then lane 31 to the upper half.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // row_bcast 15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // row_bcast 31
  return x;
}

// Sequence b0 + lane, its steps, and the steps up to and with it of those
// from b0 on.
struct LaneSeq {
  Seq s;
  int cost, incl;
};

__device__ __forceinline__ int cost_of(const Seq& s) { return s.n > 0 ? max(1, (s.len + kStep - 1) / kStep) : 0; }

__device__ __forceinline__ LaneSeq lane_seq(const KvArgs& a, int b0, int lane) {
  LaneSeq r;
  r.s = Seq{0, 0, 0};
  if (b0 + lane < a.B) r.s = seq_of(a, b0 + lane);
  r.cost = cost_of(r.s);
  r.incl = wave_scan(r.cost);
  return r;
}

// `head`: the first 64 sequences (for most steps all there are)
__device__ __forceinline__ Cut cut_of(const KvArgs& a, int workers, const LaneSeq& head, int lane) {
  Cut c;
  c.total = __builtin_amdgcn_readlane(head.incl, 63);
  if (a.B > 64) {
    int sum = 0;
    for (int b = 64 + lane; b < a.B; b += 64) sum += cost_of(seq_of(a, b));
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    c.total += __builtin_amdgcn_readfirstlane(sum);
  }
  // whole rounds of the waves, so that none idles in a range's last one
  c.per = ((c.total + workers - 1) / workers + kWaves - 1) / kWaves * kWaves;
  return c;
}

__device__ __forceinline__ Seq of_lane(const LaneSeq& r, int l) {
  return Seq{__builtin_amdgcn_readlane(r.s.len, l), __builtin_amdgcn_readlane(r.s.n, l),
             __builtin_amdgcn_readlane(r.s.row0, l)};
}

// The sequence that holds step `at` (< total), and its first step.
__device__ __forceinline__ int seq_at(const KvArgs& a, int at, LaneSeq r, int lane, int* first) {
  int before = 0;
  for (int b0 = 0;;) {
    const uint64_t past = __ballot(before + r.incl > at);
    if (past) {
      const int l = __builtin_ctzll(past);
      *first = before + __builtin_amdgcn_readlane(r.incl - r.cost, l);
      return b0 + l;
    }
    before += __builtin_amdgcn_readlane(r.incl, 63);
    b0 += 64;
    if (b0 >= a.B) return a.B;              // (not for at < total)
    r = lane_seq(a, b0, lane);
  }
}

// Sequence b (the same for the whole wave).
__device__ __forceinline__ Seq uniform_seq(const KvArgs& a, const LaneSeq& head, int b) {
  if (b < 64) return of_lane(head, b);
  const Seq s = seq_of(a, b);
  return Seq{__builtin_amdgcn_readfirstlane(s.len), __builtin_amdgcn_readfirstlane(s.n),
             __builtin_amdgcn_readfirstlane(s.row0)};
}

// Page of block blk of sequence b; blocks behind the context repeat its last.
__device__ __forceinline__ int page_at(const KvArgs& a, int len, int b, int blk) {
  return a.table[(int64_t)b * a.table_stride + (min(blk, ((len + 15) >> 4) - 1) >> a.lb)];
}

// A block's place in the cache and how many of its tokens exist; one that
// does not exist stands for the cache's first block, with no tokens.
struct BlockAt {
  int64_t at;
  int valid;
};

__device__ __forceinline__ BlockAt find_block(const KvArgs& a, int len, int hk, int blk, int page_lane) {
  const int page = __builtin_amdgcn_readfirstlane(page_lane);
  const bool there = (unsigned)page < (unsigned)a.n_pages && 16 * blk < len;
  BlockAt r;
  r.valid = there ? min(len - 16 * blk, 16) : 0;
  r.at = there ? (((int64_t)page * a.Hk + hk) << a.lb) + (blk & ((1 << a.lb) - 1)) : 0;
  return r;
}

__device__ __forceinline__ uint32_t word_of(const u32x4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

// A score's factor: scale * log2(e) times the block's scale, by its exponent,
// kept finite and above zero (0 * inf and inf * 0 are no scores).
__device__ __forceinline__ float score_factor(float c, float block_scale) {
  const float e = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, block_scale) & 0x7F800000u);
  return fminf(fmaxf(c * e, 0x1p-126f), 0x1.fffffep127f);
}

// Codes are read once, so they need not displace what the caches hold.
__device__ __forceinline__ u32x4 load_codes(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Workgroups of a compute unit that the registers leave room for.
constexpr int occupancy(int dim, int nr) { return dim > 128 ? 1 : nr == 1 ? 3 : 2; }

// Outputs are summed 2^-32 times their size: a block's largest value, 448 *
// 2^121, lies outside of 32-bit and bf16 numbers, and where its token is
// masked 0 * inf would spoil the row.
constexpr float kVDown = 0x1p-32f, kVUp = 0x1p32f;

// Workgroup: one range, one key head, up to 16*NR rows of each of its
// sequences (row r = token r / group, query head r % group of the key head's
// group).  Within a segment each wave takes every fourth step and keeps its
// own running maximum, sum and output, joined over the waves at the end.
//
// With K as the first operand a 16x16x32 product gives a lane 4 positions of
// one row (column lane % 16), which is what the second product takes as its
// operand after exp, so the weights never leave the registers; the cache's
// layout gives K and V codes in operand order by 16-byte loads.  The operands
// are exact: K's are the codes themselves, their scale in the score's factor,
// V's are bf16 numbers whatever the row type is (fp16 ends at 65504, and a code
// times its scale does not), and a weight is the sum of two bf16 numbers, its
// rounded value and what that leaves, good to 2^-16.  (One product of rounded
// weights: 777 positions 6.6 us a call, 6.9 with both, 8 contexts of 16384, 32
// tokens each, heads of 128, 135 and 153, long contexts the same; bf16 outputs
// were then 0.0021 to 0.0024 of their size off, 0.0017 with both, which is their
// own rounding.)
// HBM bounds it, so a wave's loads never stop: the next step's K codes are asked
// for as soon as this step's are in the first product, its V codes after the
// second.  (Two steps ahead holds twice the registers and gains nothing: 16
// drafts of up to 3 tokens 28.2 us a call where one step took 26.0.)
//
// One context of 131071, 8 key heads of 128: 269 MB in 45 us, 6.0 TB/s; 64 of
// up to 8192: 603 MB in 99 us, 6.1 TB/s (the copy reaches 4.7, reading and
// writing).  16 drafts of up to 3 tokens, 64 + 8 heads, contexts up to 4099: 85
// MB in 23 us: five rounds a wave, each of its steps' latencies one after the
// other, and what comes before the first.
//
// Short: a workgroup of 8 waves takes a whole sequence, so that there is no
// join to launch (768 positions, 8 key heads: 6.8 us a call, parts and join 7.9).
template <typename T, int D, int NR, bool Short>
__global__ __launch_bounds__(64 * (Short ? kShortWaves : kWaves), Short ? 1 : occupancy(D, NR)) void decode_kernel(DecodeArgs a) {
  constexpr int NW = Short ? kShortWaves : kWaves;
  constexpr int kKb = D / 32;               // k-blocks of a score
  constexpr int kDt = D / 16;               // 16-column tiles of the output
  constexpr int kP = D / 64;                // pieces of a block's K, of its V
  __shared__ float so[NW][16][D + 4];
  __shared__ float sm[NW][16], sl[NW][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int hk = blockIdx.x, worker = blockIdx.y;
  const int group = a.Hq / a.kv.Hk;
  const int r0 = blockIdx.z * 16 * NR;

  LaneSeq head{};
  Cut cut{};
  int pos, end, first, b;
  if (Short) {
    b = worker;
    first = pos = 0;
    end = 0x7FFFFFFF;
  } else {
    head = lane_seq(a.kv, 0, lane);
    cut = cut_of(a.kv, a.split.n, head, lane);
    pos = worker * cut.per;
    end = min(pos + cut.per, cut.total);
    if (pos >= end) return;                 // the whole workgroup
    b = seq_at(a.kv, pos, head, lane, &first);
  }

  for (bool again = false; pos < end && b < a.kv.B; ++b) {
    const Seq s = Short ? seq_of(a.kv, b) : uniform_seq(a.kv, head, b);
    const int steps = (s.len + kStep - 1) / kStep, cost = cost_of(s);
    const int s0 = pos - first, s1 = min(min(end - first, cost), steps);
    const bool whole = Short || (pos == first && first + cost <= end);
    // the range with a sequence's first step tells the join where its parts lie
    if (!Short && a.split.n > 1 && pos == first && cost > 0 && hk == 0 && blockIdx.z == 0 && threadIdx.x == 0)
      a.split.where[b] = make_int2(worker, (first + cost - 1) / cut.per - worker + 1);
    first += cost;
    pos = Short ? end : min(first, end);
    const int rows = min(s.n, a.kv.max_new) * group;
    if (r0 >= rows) continue;               // (the same for the whole workgroup)

    // this lane's row of each row tile: its q (the second operand) and the
    // last position it sees
    u32x4 q[NR][kKb];
    int last[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const int r = r0 + 16 * t + n16;
      const int i = r / group, gh = r % group;
      last[t] = r < rows ? s.len - s.n + i : -1;
#pragma unroll
      for (int k = 0; k < kKb; ++k) q[t][k] = u32x4{0, 0, 0, 0};
      if (r < rows) {
        const uint16_t* p = (const uint16_t*)a.q + (int64_t)(s.row0 + i) * a.qs + (int64_t)(hk * group + gh) * D + 8 * g;
#pragma unroll
        for (int k = 0; k < kKb; ++k) q[t][k] = *reinterpret_cast<const u32x4*>(p + 32 * k);
      }
    }
    const int first_last = s.len - s.n + r0 / group;   // what the first row sees: all rows see up to it

    float m[NR], l[NR];
    f32x4 o[NR][kDt];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      m[t] = kMinusInf;
      l[t] = 0.f;
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    int st = s0 + wave;
    if (st < s1) {
      u32x4 kr[2][kP], vr[2][kP];
      float2 sc2[2];
      BlockAt cur[2];
      int page[2], first_page[2];           // pages of the next step
#pragma unroll
      for (int i = 0; i < 2; ++i) first_page[i] = page_at(a.kv, s.len, b, 2 * st + i);
#pragma unroll
      for (int i = 0; i < 2; ++i) page[i] = page_at(a.kv, s.len, b, 2 * (st + NW) + i);
#pragma unroll
      for (int i = 0; i < 2; ++i) cur[i] = find_block(a.kv, s.len, hk, 2 * st + i, first_page[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* p = a.kv.codes + cur[i].at * (32 * D) + 16 * lane;
        sc2[i] = *reinterpret_cast<const float2*>(a.kv.scales + 2 * cur[i].at);
#pragma unroll
        for (int k = 0; k < kP; ++k) kr[i][k] = load_codes(p + 1024 * k);
#pragma unroll
        for (int k = 0; k < kP; ++k) vr[i][k] = load_codes(p + 16 * D + 1024 * k);
      }
      for (; st < s1; st += NW) {
        // scores (of codes, without the scales): position 32 st + 16 i + 4 g + j in sc[t][i][j]
        f32x4 sc[NR][2];
        float ck[2], sv[2];
        int valid[2];
#pragma unroll
        for (int t = 0; t < NR; ++t) sc[t][0] = sc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          valid[i] = cur[i].valid;
          ck[i] = score_factor(a.c, valid[i] ? sc2[i].x : 1.f);
          sv[i] = valid[i] ? sc2[i].y * kVDown : 1.f;
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const u32x4 ka = dec8<T>(kr[i][p].x, kr[i][p].y, 1.f), kb = dec8<T>(kr[i][p].z, kr[i][p].w, 1.f);
#pragma unroll
            for (int t = 0; t < NR; ++t) {
              sc[t][i] = T::mma16(ka, q[t][2 * p], sc[t][i]);
              sc[t][i] = T::mma16(kb, q[t][2 * p + 1], sc[t][i]);
            }
          }
        }
        // the next step's K (in the last step: this one's again, so that the
        // number of loads under way is the same on every path)
        const bool more = st + NW < s1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (more) cur[i] = find_block(a.kv, s.len, hk, 2 * (st + NW) + i, page[i]);
          const uint8_t* p = a.kv.codes + cur[i].at * (32 * D) + 16 * lane;
          sc2[i] = *reinterpret_cast<const float2*>(a.kv.scales + 2 * cur[i].at);
#pragma unroll
          for (int k = 0; k < kP; ++k) kr[i][k] = load_codes(p + 1024 * k);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) page[i] = page_at(a.kv, s.len, b, 2 * (st + 2 * NW) + i);
        const bool all = valid[0] == 16 && valid[1] == 16 && kStep * st + kStep - 1 <= first_last;
        bool bad_v = false;                 // a code for not a number among V's valid tokens
        if (!all) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool there = 4 * g + j < valid[i];
              const int at = kStep * st + 16 * i + 4 * g + j;
#pragma unroll
              for (int t = 0; t < NR; ++t)
                if (!there || at > last[t]) sc[t][i][j] = kMinusInf;
            }
            // V of tokens that are not there becomes zero: 0 * NaN would spoil the sum
            const int nv = min(max(valid[i] - 4 * g, 0), 4);
            const uint32_t keep = nv >= 4 ? 0xFFFFFFFFu : (1u << (8 * nv)) - 1u;
#pragma unroll
            for (int p = 0; p < kP; ++p) {
              vr[i][p] &= u32x4{keep, keep, keep, keep};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t x = word_of(vr[i][p], w) & 0x7F7F7F7Fu;
                bad_v |= ((x + 0x01010101u) & 0x80808080u) != 0;
              }
            }
          }
          bad_v = __any(bad_v);
        }
        u32x4 hi[NR], lo[NR];
#pragma unroll
        for (int t = 0; t < NR; ++t) {
          // powers of two under the running maximum, which is raised only when a
          // score exceeds it by 2^8 (or a row has none yet), so that the sums are
          // hardly ever rescaled; the weights are then up to 2^8, and their two
          // roundings relative to themselves
          const float base = m[t] == kMinusInf ? 0.f : m[t];
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __builtin_fmaf(sc[t][j >> 2][j & 3], ck[j >> 2], -base);
          float mx = fmaxf(fmaxf(x[0], x[1]), x[2]);
          mx = fmaxf(fmaxf(mx, x[3]), x[4]);
          mx = fmaxf(fmaxf(mx, x[5]), x[6]);
          mx = max_rows4(fmaxf(mx, x[7]));
          const bool raise = mx > kLazy || (m[t] == kMinusInf && mx > kMinusInf);
          if (__any(raise)) {
            // from the scores again: under a maximum far below them x has lost bits
            float top = kMinusInf;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, sc[t][j >> 2][j & 3] * ck[j >> 2]);
            top = max_rows4(top);
            const float r = !raise ? 1.f : m[t] == kMinusInf ? 0.f : exp2_fast(m[t] - top);
            if (raise) m[t] = top;
            l[t] *= r;
#pragma unroll
            for (int k = 0; k < kDt; ++k) o[t][k] *= r;
            const float now = raise ? top : base;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __builtin_fmaf(sc[t][j >> 2][j & 3], ck[j >> 2], -now);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = exp2_fast(x[j]);
            l[t] += x[j];
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint32_t h = Bf16::cvt2(x[j], x[j + 1]);
            hi[t][j >> 1] = h;
            lo[t][j >> 1] = Bf16::cvt2(x[j] - Bf16::lo(h), x[j + 1] - Bf16::hi(h));
          }
        }
        // a valid V that is not a number, behind some rows' last position: take
        // it out of the product, and give it to the rows that see it
        if (bad_v) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
              uint32_t clean[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t v = word_of(vr[i][p], w);
                const uint32_t isnan = (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;   // bytes 0 or 1
                clean[w] = v & ~(isnan * 255u);
                // the word's column is 64 p + 16 w + lane % 16; the output's lane
                // holds columns 16 dt + 4 g + 0..3 of row lane % 16
                for (uint64_t lanes = __ballot(isnan != 0); lanes; lanes &= lanes - 1) {
                  const int k = __builtin_ctzll(lanes);
                  const uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)isnan, k);
                  const int col = k & 15, at = kStep * st + 16 * i + 4 * (k >> 4);
#pragma unroll
                  for (int t = 0; t < NR; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      if (((bits >> (8 * j)) & 1) && at + j <= last[t] && (col >> 2) == g) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                          if ((col & 3) == e) o[t][4 * p + w][e] = __builtin_nanf("");
                      }
                }
              }
              vr[i][p] = u32x4{clean[0], clean[1], clean[2], clean[3]};
            }
          }
        }
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          u32x4 v[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t w0 = word_of(vr[0][p], w), w1 = word_of(vr[1][p], w);
            v[w].x = Bf16::dec2(w0, sv[0], false);
            v[w].y = Bf16::dec2(w0, sv[0], true);
            v[w].z = Bf16::dec2(w1, sv[1], false);
            v[w].w = Bf16::dec2(w1, sv[1], true);
#pragma unroll
            for (int t = 0; t < NR; ++t) o[t][4 * p + w] = Bf16::mma16(v[w], hi[t], o[t][4 * p + w]);
          }
#pragma unroll
          for (int t = 0; t < NR; ++t)
#pragma unroll
            for (int w = 0; w < 4; ++w) o[t][4 * p + w] = Bf16::mma16(v[w], lo[t], o[t][4 * p + w]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* p = a.kv.codes + cur[i].at * (32 * D) + 16 * D + 16 * lane;
#pragma unroll
          for (int k = 0; k < kP; ++k) vr[i][k] = load_codes(p + 1024 * k);
        }
      }
    }

    // join the waves: row n16, columns 16 d + 4 g + j of o[t][d][j]
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const float lt = sum_rows4(l[t]);
      if (t || again) __syncthreads();
      again = true;
      if (g == 0) {
        sm[wave][n16] = m[t];
        sl[wave][n16] = lt;
      }
#pragma unroll
      for (int d = 0; d < kDt; ++d) *reinterpret_cast<f32x4*>(&so[wave][n16][16 * d + 4 * g]) = o[t][d];
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * NW) {
        const int row = i / (D / 4), ch = i % (D / 4);
        const int r = r0 + 16 * t + row;
        if (r >= rows) continue;
        float mx = kMinusInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[w][row]);
        const float base = mx == kMinusInf ? 0.f : mx;
        float sum = 0.f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          // (a wave that saw nothing has maximum -inf and zeros)
          const float e = exp2_fast(sm[w][row] - base);
          sum += e * sl[w][row];
          acc += *reinterpret_cast<const f32x4*>(&so[w][row][4 * ch]) * e;
        }
        const int tok = r / group, h = hk * group + r % group;
        if (!whole) {
          const int64_t at = ((int64_t)(worker + b) * a.kv.max_new + tok) * a.Hq + h;
          *reinterpret_cast<f32x4*>(a.split.o + at * D + 4 * ch) = acc;
          if (ch == 0) *reinterpret_cast<float2*>(a.split.ml + 2 * at) = make_float2(mx, sum);
        } else {
          const float inv = sum == 0.f ? 0.f : kVUp / sum;
          u32x2 w;
          w.x = T::cvt2(acc[0] * inv, acc[1] * inv);
          w.y = T::cvt2(acc[2] * inv, acc[3] * inv);
          const int64_t row_at = s.row0 + tok;
          *reinterpret_cast<u32x2*>((uint16_t*)a.out + row_at * a.os + (int64_t)h * D + 4 * ch) = w;
          if (ch == 0 && a.lse) a.lse[row_at * a.Hq + h] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
        }
      }
    }
  }
}

// Joins the parts of one row and head: a workgroup each.  Its threads take a
// part's columns, 4 each, of 256 / (D/4) parts at once: latency is what
// counts.  32 rows of 96 parts, heads of 128: 5 us.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(DecodeArgs a) {
  constexpr int kCh = D / 4, kAtOnce = kThreads / kCh;
  __shared__ f32x4 acc_s[kAtOnce][kCh];
  __shared__ float sum_s[kAtOnce];
  const int lane = threadIdx.x & 63;
  const int b = blockIdx.x / a.kv.max_new, i = blockIdx.x % a.kv.max_new, h = blockIdx.y;
  const int2 where = a.split.where[b];      // (nothing was written for a sequence without rows)
  const Seq s = seq_rows(a.kv.cu, a.kv.per_seq, a.kv.T, b, a.kv.codes);
  if (i >= s.n) return;
  const int w0 = where.x, n = where.y;
  if (n == 1) return;                       // written by the range that holds it
  const int64_t pitch = (int64_t)a.kv.max_new * a.Hq, at = (w0 + b) * pitch + (int64_t)i * a.Hq + h;
  const float2* ml = reinterpret_cast<const float2*>(a.split.ml) + at;
  float mx = kMinusInf;
  for (int p = lane; p < n; p += 64) mx = fmaxf(mx, ml[p * pitch].x);
  for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  const float base = mx == kMinusInf ? 0.f : mx;
  const int ch = threadIdx.x % kCh, p0 = threadIdx.x / kCh;
  float sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = p0; p < n; p += kAtOnce) {
    const float2 v = ml[p * pitch];
    const float e = exp2_fast(v.x - base);  // (a part that saw nothing: maximum -inf, zeros)
    sum += e * v.y;
    acc += *reinterpret_cast<const f32x4*>(a.split.o + (at + p * pitch) * D + 4 * ch) * e;
  }
  acc_s[p0][ch] = acc;
  if (ch == 0) sum_s[p0] = sum;
  __syncthreads();
  if (p0 != 0) return;
#pragma unroll
  for (int p = 1; p < kAtOnce; ++p) {
    acc += acc_s[p][ch];
    sum += sum_s[p];
  }
  const float inv = sum == 0.f ? 0.f : kVUp / sum;
  u32x2 w;
  w.x = T::cvt2(acc[0] * inv, acc[1] * inv);
  w.y = T::cvt2(acc[2] * inv, acc[3] * inv);
  const int64_t row = s.row0 + i;
  *reinterpret_cast<u32x2*>((uint16_t*)a.out + row * a.os + (int64_t)h * D + 4 * ch) = w;
  if (ch == 0 && a.lse) a.lse[row * a.Hq + h] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The same by a wave each, four heads a workgroup: a few parts.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void join_few_kernel(DecodeArgs a) {
  const int b = blockIdx.x / a.kv.max_new, i = blockIdx.x % a.kv.max_new, h = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  const int2 where = a.split.where[b];
  const Seq s = seq_rows(a.kv.cu, a.kv.per_seq, a.kv.T, b, a.kv.codes);
  if (h >= a.Hq || i >= s.n || where.y == 1) return;
  const int64_t pitch = (int64_t)a.kv.max_new * a.Hq, at = (where.x + b) * pitch + (int64_t)i * a.Hq + h, row = s.row0 + i;
  join_row<T, D>(a.split.o + at * D, a.split.ml + 2 * at, where.y, pitch, (uint16_t*)a.out + row * a.os + (int64_t)h * D,
                 a.lse ? a.lse + row * a.Hq + h : nullptr, kVUp, threadIdx.x & 63);
}

int rows_of(const KvArgs& kv, int Hq) { return kv.max_new * (Hq / kv.Hk); }

// Row tiles of 16 a workgroup takes: two serve up to 32 rows with one read of
// the codes and leave room for two workgroups a compute unit.  More rows go to
// neighbours in the grid's third dimension, which find the codes in the
// caches: 8 contexts of 16384, 32 tokens each, 32 + 8 heads of 64, 118 us (one
// tile a workgroup 146); heads of 128 153 us (252).  (Four tiles, at one workgroup
// a compute unit, were no better.)
int row_tiles(const KvArgs& kv, int Hq) { return rows_of(kv, Hq) <= 16 ? 1 : 2; }

// Whether contexts (by the page table) are taken whole: up to six rounds of a
// workgroup's waves, or four where the workgroups would leave most of the card
// idle (us a call whole, and cut into parts and joined; 32 + 8 heads of 128, of
// 1024, 1280 and 1536 positions: one sequence 7.8, 8.9, 10.0 and 7.9, 8.2, 8.3; four
// 7.9, 9.1, 10.0 and 8.4, 9.8, 10.4; 16 8.5, 10.1, 11.6 and 11.4, 13.6, 14.6).  Two
// tiles of the widest rows do not fit the registers of 8 waves.
bool is_short(const KvArgs& kv, int nr) {
  const int rounds = (int64_t)kv.B * kv.Hk >= 32 ? 6 : 4;
  return kv.max_len <= rounds * kShortWaves * kStep && nr * kv.D <= 256 && kv.B <= 65535;
}

template <typename T, int D>
void (*pick(int nr, bool shrt))(DecodeArgs) {
  if (nr == 1) return shrt ? decode_kernel<T, D, 1, true> : decode_kernel<T, D, 1, false>;
  return shrt ? decode_kernel<T, D, (D > 128 ? 1 : 2), true> : decode_kernel<T, D, 2, false>;
}

template <typename T>
void (*pick_dim(int dim, int nr, bool shrt))(DecodeArgs) {
  return dim == 64 ? pick<T, 64>(nr, shrt) : dim == 128 ? pick<T, 128>(nr, shrt) : pick<T, 256>(nr, shrt);
}

template <typename T>
void (*pick_join(int dim, bool few))(DecodeArgs) {
  if (dim == 64) return few ? join_few_kernel<T, 64> : join_kernel<T, 64>;
  if (dim == 128) return few ? join_few_kernel<T, 128> : join_kernel<T, 128>;
  return few ? join_few_kernel<T, 256> : join_kernel<T, 256>;
}

}  // namespace

namespace qmoe {

int attn_decode_workers(const KvArgs& kv, int Hq, int cus) {
  const int nr = row_tiles(kv, Hq);
  if (is_short(kv, nr)) return 1;
  const int64_t wgs = (int64_t)kv.Hk * ((rows_of(kv, Hq) + 16 * nr - 1) / (16 * nr));
  const int64_t most = kv.B * (((int64_t)kv.max_len + kStep * kWaves - 1) / (kStep * kWaves));
  int64_t n = (int64_t)occupancy(kv.D, nr) * cus / wgs;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

hipError_t launch_attn_decode(const DecodeArgs& a, int dtype, hipStream_t s) {
  const int nr = row_tiles(a.kv, a.Hq);
  const bool bf = dtype == 0, shrt = is_short(a.kv, nr);
  auto fn = bf ? pick_dim<Bf16>(a.kv.D, nr, shrt) : pick_dim<F16>(a.kv.D, nr, shrt);
  hipLaunchKernelGGL(fn, dim3((unsigned)a.kv.Hk, (unsigned)(shrt ? a.kv.B : a.split.n),
                              (unsigned)((rows_of(a.kv, a.Hq) + 16 * nr - 1) / (16 * nr))),
                     dim3(64 * (shrt ? kShortWaves : kWaves)), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.split.n == 1) return e;
  // a wave a row where the ranges make at most 16 parts a sequence (16 users'
  // drafts of 3, 64 heads, 4 parts: 3.9 us, a workgroup a row 5.5)
  const bool few = a.split.n <= 16 * a.kv.B;
  auto join = bf ? pick_join<Bf16>(a.kv.D, few) : pick_join<F16>(a.kv.D, few);
  hipLaunchKernelGGL(join, dim3((unsigned)(a.kv.B * (int64_t)a.kv.max_new), (unsigned)(few ? (a.Hq + 3) / 4 : a.Hq)),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe

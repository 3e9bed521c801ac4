// Attention of a few new tokens of each sequence over its cached context
// (moe_attn_decode), and the join of parts of a context.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.hpp"

using namespace qmoe;
using namespace qmoe_dev;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kStep = 32;                   // positions a wave takes at once: two blocks

// The parts' share of a context: its steps of 32 positions, dealt out in
// groups of kWaves steps (one step a wave), the first parts first.
__device__ __forceinline__ int steps_per_part(int steps, int n_split) {
  return (((steps + n_split - 1) / n_split) + kWaves - 1) / kWaves * kWaves;
}

// One block of the context as a wave holds it.
template <int D>
struct BlockRegs {
  u32x4 k[D / 64], v[D / 64];
  float sk, sv;
  int valid;                                // tokens of it that exist
};

template <int D>
__device__ __forceinline__ void load_block(const KvArgs& a, const Seq& s, int b, int hk, int blk, int lane,
                                           BlockRegs<D>* r) {
  const int nblk = (s.len + 15) >> 4;
  const int64_t at = blk < nblk ? block_of(a, b, blk, hk) : -1;
  r->valid = at < 0 ? 0 : min(s.len - 16 * blk, 16);
  const int64_t i = at < 0 ? 0 : at;        // (there is always a first block to read)
  const uint8_t* p = a.codes + i * (32 * D) + 16 * lane;
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    r->k[q] = *reinterpret_cast<const u32x4*>(p + 1024 * q);
    r->v[q] = *reinterpret_cast<const u32x4*>(p + 16 * D + 1024 * q);
  }
  const float2 sc = *reinterpret_cast<const float2*>(a.scales + 2 * i);
  r->sk = at < 0 ? 1.f : sc.x;
  r->sv = at < 0 ? 1.f : sc.y;
}

__device__ __forceinline__ uint32_t word_of(const u32x4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

// Workgroup: one part of the context of one sequence and key head, up to
// 16*NR of its rows (row r = token r / group, query head r % group of the key
// head's group).  Each wave takes every fourth step of 32 positions and
// keeps its own running maximum, sum and output, joined over the waves at
// the end.  With K as the first operand a 16x16x32 product gives a lane 4
// positions of one row (column lane % 16), which is what the second product
// takes as its operand after exp, so the weights never leave the registers;
// the cache's layout gives K and V codes in operand order by 16-byte loads.
template <typename T, int D, int NR>
__global__ __launch_bounds__(kThreads) void decode_kernel(DecodeArgs a) {
  constexpr int kKb = D / 32;               // k-blocks of a score
  constexpr int kDt = D / 16;               // 16-column tiles of the output
  __shared__ float so[kWaves][16][D + 4];
  __shared__ float sm[kWaves][16], sl[kWaves][16];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int part = blockIdx.y;
  const int b = blockIdx.x / a.kv.Hk, hk = blockIdx.x % a.kv.Hk;
  const int group = a.Hq / a.kv.Hk;
  const Seq s = seq_of(a.kv, b);
  const int r0 = blockIdx.z * 16 * NR;
  const int rows = s.n * group;
  if (r0 >= rows) return;                   // the whole workgroup

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
  const int first_last = s.len - s.n + r0 / group;     // what the first row sees: all rows see up to it

  float m[NR], l[NR];
  f32x4 o[NR][kDt];
#pragma unroll
  for (int t = 0; t < NR; ++t) {
    m[t] = kMinusInf;
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < kDt; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int steps = (s.len + kStep - 1) / kStep;
  const int per = steps_per_part(steps, a.split.n);
  const int s0 = part * per, s1 = min(s0 + per, steps);

  for (int st = s0 + wave; st < s1; st += kWaves) {
    BlockRegs<D> B0, B1;
    load_block<D>(a.kv, s, b, hk, 2 * st, lane, &B0);
    load_block<D>(a.kv, s, b, hk, 2 * st + 1, lane, &B1);
    // scores: position 32 st + 16 i + 4 g + j in sc[t][i][j]
    f32x4 sc[NR][2];
#pragma unroll
    for (int t = 0; t < NR; ++t) sc[t][0] = sc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const BlockRegs<D>& Bl = i ? B1 : B0;
        const u32x4 ka = dec8<T>(Bl.k[p].x, Bl.k[p].y, Bl.sk), kb = dec8<T>(Bl.k[p].z, Bl.k[p].w, Bl.sk);
#pragma unroll
        for (int t = 0; t < NR; ++t) {
          sc[t][i] = T::mma16(ka, q[t][2 * p], sc[t][i]);
          sc[t][i] = T::mma16(kb, q[t][2 * p + 1], sc[t][i]);
        }
      }
    }
    const bool all = B0.valid == 16 && B1.valid == 16 && kStep * st + kStep - 1 <= first_last;
    bool bad_v = false;                     // a code for not a number among V's valid tokens
    if (!all) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        BlockRegs<D>& Bl = i ? B1 : B0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool there = 4 * g + j < Bl.valid;
          const int pos = kStep * st + 16 * i + 4 * g + j;
#pragma unroll
          for (int t = 0; t < NR; ++t)
            if (!there || pos > last[t]) sc[t][i][j] = kMinusInf;
        }
        // V of tokens that are not there becomes zero: 0 * NaN would spoil the sum
        const int nv = min(max(Bl.valid - 4 * g, 0), 4);
        const uint32_t keep = nv >= 4 ? 0xFFFFFFFFu : (1u << (8 * nv)) - 1u;
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
          Bl.v[p] &= u32x4{keep, keep, keep, keep};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = word_of(Bl.v[p], w) & 0x7F7F7F7Fu;
            bad_v |= ((x + 0x01010101u) & 0x80808080u) != 0;
          }
        }
      }
      bad_v = __any(bad_v);
    }
    u32x4 pk[NR];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = sc[t][j >> 2][j & 3] * a.c;
      float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      mx = fmaxf(m[t], max_rows4(mx));
      if (__any(mx > m[t])) {
        const float r = m[t] == kMinusInf ? 0.f : exp2_fast(m[t] - mx);
        l[t] *= r;
#pragma unroll
        for (int d = 0; d < kDt; ++d) o[t][d] *= r;
        m[t] = mx;
      }
      const float base = mx == kMinusInf ? 0.f : mx;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = exp2_fast(x[j] - base);
        l[t] += x[j];
      }
      pk[t].x = T::cvt2(x[0], x[1]);
      pk[t].y = T::cvt2(x[2], x[3]);
      pk[t].z = T::cvt2(x[4], x[5]);
      pk[t].w = T::cvt2(x[6], x[7]);
    }
    // a valid V that is not a number, behind some rows' last position: take
    // it out of the product, and give it to the rows that see it
    if (bad_v) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        BlockRegs<D>& Bl = i ? B1 : B0;
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
          uint32_t clean[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t v = word_of(Bl.v[p], w);
            const uint32_t isnan = (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;   // bytes 0 or 1
            clean[w] = v & ~(isnan * 255u);
            // the word's column is 64 p + 16 w + lane % 16; the output's lane
            // holds columns 16 dt + 4 g + 0..3 of row lane % 16
            for (uint64_t lanes = __ballot(isnan != 0); lanes; lanes &= lanes - 1) {
              const int k = __builtin_ctzll(lanes);
              const uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)isnan, k);
              const int col = k & 15, pos0 = kStep * st + 16 * i + 4 * (k >> 4);
#pragma unroll
              for (int t = 0; t < NR; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (((bits >> (8 * j)) & 1) && pos0 + j <= last[t] && (col >> 2) == g) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if ((col & 3) == e) o[t][4 * p + w][e] = __builtin_nanf("");
                  }
            }
          }
          Bl.v[p] = u32x4{clean[0], clean[1], clean[2], clean[3]};
        }
      }
    }
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t w0 = word_of(B0.v[p], w), w1 = word_of(B1.v[p], w);
        u32x4 v;
        v.x = T::dec2(w0, B0.sv, false);
        v.y = T::dec2(w0, B0.sv, true);
        v.z = T::dec2(w1, B1.sv, false);
        v.w = T::dec2(w1, B1.sv, true);
#pragma unroll
        for (int t = 0; t < NR; ++t) o[t][4 * p + w] = T::mma16(v, pk[t], o[t][4 * p + w]);
      }
    }
  }

  // join the waves: row n16, columns 16 d + 4 g + j of o[t][d][j]
#pragma unroll
  for (int t = 0; t < NR; ++t) {
    const float lt = sum_rows4(l[t]);
    if (t) __syncthreads();
    if (g == 0) {
      sm[wave][n16] = m[t];
      sl[wave][n16] = lt;
    }
#pragma unroll
    for (int d = 0; d < kDt; ++d) *reinterpret_cast<f32x4*>(&so[wave][n16][16 * d + 4 * g]) = o[t][d];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 4); i += kThreads) {
      const int row = i / (D / 4), ch = i % (D / 4);
      const int r = r0 + 16 * t + row;
      if (r >= rows) continue;
      float mx = kMinusInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, sm[w][row]);
      const float base = mx == kMinusInf ? 0.f : mx;
      float sum = 0.f;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        // (a wave that saw nothing has maximum -inf and zeros)
        const float e = exp2_fast(sm[w][row] - base);
        sum += e * sl[w][row];
        acc += *reinterpret_cast<const f32x4*>(&so[w][row][4 * ch]) * e;
      }
      const int tok = s.row0 + r / group, h = hk * group + r % group;
      if (a.split.n > 1) {
        const int64_t at = ((int64_t)part * a.kv.T + tok) * a.Hq + h;
        *reinterpret_cast<f32x4*>(a.split.o + at * D + 4 * ch) = acc;
        if (ch == 0) *reinterpret_cast<float2*>(a.split.ml + 2 * at) = make_float2(mx, sum);
      } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        u32x2 w;
        w.x = T::cvt2(acc[0] * inv, acc[1] * inv);
        w.y = T::cvt2(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<u32x2*>((uint16_t*)a.out + (int64_t)tok * a.os + (int64_t)h * D + 4 * ch) = w;
        if (ch == 0 && a.lse) a.lse[(int64_t)tok * a.Hq + h] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
      }
    }
  }
}

// Joins the parts of one row and head: a wave each.
template <typename T>
__global__ __launch_bounds__(kThreads) void join_kernel(JoinArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int h = blockIdx.y * kWaves + wave;
  if (h >= a.Hq) return;
  const int b = blockIdx.x / a.max_new, i = blockIdx.x % a.max_new;
  const Seq s = seq_rows(a.cu, a.per_seq, a.T, b);
  if (i >= s.n) return;
  const int tok = s.row0 + i;
  const int64_t at = (int64_t)tok * a.Hq + h, pitch = (int64_t)a.T * a.Hq;
  float mx = kMinusInf;
  for (int p = lane; p < a.split.n; p += 64) mx = fmaxf(mx, a.split.ml[2 * (p * pitch + at)]);
  for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  const float base = mx == kMinusInf ? 0.f : mx;
  float sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const bool on = 4 * lane < a.D;
  for (int p = 0; p < a.split.n; ++p) {
    const float2 ml = *reinterpret_cast<const float2*>(a.split.ml + 2 * (p * pitch + at));
    if (ml.x == kMinusInf) continue;        // an empty part's sums are not read
    const float e = exp2_fast(ml.x - base);
    sum += e * ml.y;
    if (on) acc += *reinterpret_cast<const f32x4*>(a.split.o + (p * pitch + at) * a.D + 4 * lane) * e;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (on) {
    u32x2 w;
    w.x = T::cvt2(acc[0] * inv, acc[1] * inv);
    w.y = T::cvt2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<u32x2*>((uint16_t*)a.out + (int64_t)tok * a.os + (int64_t)h * a.D + 4 * lane) = w;
  }
  if (lane == 0 && a.lse) a.lse[at] = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Row tiles of 16 a workgroup takes: as many as the step needs, up to 4 (64
// rows), so that the context is read once for all of them.
int row_tiles(const KvArgs& kv, int Hq) {
  const int64_t rows = (int64_t)(kv.cu ? kv.max_new : kv.per_seq) * (Hq / kv.Hk);
  return rows <= 16 ? 1 : rows <= 32 || kv.D > 128 ? 2 : 4;
}

template <typename T, int D>
void (*pick(int nr))(DecodeArgs) {
  return nr == 1 ? decode_kernel<T, D, 1> : nr == 2 ? decode_kernel<T, D, 2> : decode_kernel<T, D, (D > 128 ? 2 : 4)>;
}

}  // namespace

namespace qmoe {

int attn_decode_splits(const KvArgs& kv, int Hq, int cus) {
  const int nr = row_tiles(kv, Hq);
  const int64_t rows = (int64_t)(kv.cu ? kv.max_new : kv.per_seq) * (Hq / kv.Hk);
  const int64_t wgs = (int64_t)kv.B * kv.Hk * ((rows + 16 * nr - 1) / (16 * nr));
  const int64_t most = (kv.max_len + kStep * kWaves - 1) / (kStep * kWaves);
  int64_t n = (4ll * cus + wgs - 1) / wgs;
  if (n > most) n = most;
  if (n > 1024) n = 1024;
  return n < 1 ? 1 : (int)n;
}

hipError_t launch_attn_decode(const DecodeArgs& a, int dtype, hipStream_t s) {
  const int nr = row_tiles(a.kv, a.Hq);
  const int64_t rows = (int64_t)(a.kv.cu ? a.kv.max_new : a.kv.per_seq) * (a.Hq / a.kv.Hk);
  void (*fn)(DecodeArgs) = nullptr;
  const bool bf = dtype == 0;
  switch (a.kv.D) {
    case 64: fn = bf ? pick<Bf16, 64>(nr) : pick<F16, 64>(nr); break;
    case 128: fn = bf ? pick<Bf16, 128>(nr) : pick<F16, 128>(nr); break;
    default: fn = bf ? pick<Bf16, 256>(nr) : pick<F16, 256>(nr); break;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.kv.B * (int64_t)a.kv.Hk), (unsigned)a.split.n, (unsigned)((rows + 16 * nr - 1) / (16 * nr))),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attn_join(const JoinArgs& a, int dtype, hipStream_t s) {
  auto fn = dtype == 0 ? join_kernel<Bf16> : join_kernel<F16>;
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.B * (int64_t)a.max_new), (unsigned)((a.Hq + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe

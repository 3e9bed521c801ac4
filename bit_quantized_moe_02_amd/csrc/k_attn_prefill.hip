// Attention of packed prompts (moe_attn_prefill).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.hpp"

using namespace qmoe;
using namespace qmoe_dev;

namespace {

constexpr int kTile = 64;                   // keys a workgroup stages at once
constexpr int kWaves = 4;
// A row's weights are powers of two above a reference.  It is put 2^kHead under
// the largest score so far, and raised only when a score would exceed it by 2^kMost:
// the sums are hardly ever rescaled, and weights stay in fp16's range (up to 65504)
// while its smallest number, 2^-24, is at most 2^-34 of the row's largest weight
// (with a reference at the maximum itself, 2^-24: 4000 keys 2^-24.4 beside one that has
// no value were a third off).
constexpr float kHead = 10.f, kMost = 15.f;
constexpr int kThreads = 64 * kWaves;

// K and V rows lie in LDS as they do in memory, 2*D bytes each, their
// 16-byte pieces permuted so that the reads below spread over all banks:
// K reads take one piece of 32 different rows, V reads (transposing) 64
// bytes of 8 rows.
template <int D>
__device__ __forceinline__ int k_piece(int row, int piece) {
  return D == 64 ? piece ^ ((row >> 1) & 7) : piece ^ (row & 15);
}
template <int D>
__device__ __forceinline__ int v_piece(int row, int piece) {
  return D == 64 ? piece ^ (4 * ((row >> 1) & 1)) : piece ^ (4 * (row & 3));
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// x, computed here and not before the loop: what only rare branches need
// must not hold registers through the loop.
__device__ __forceinline__ int only_here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Copies tiles of keys into LDS: 1024 bytes an instruction, which go there in
// lane order, so the permutation is in what each lane reads.  The reads go
// through a buffer descriptor that ends behind the sequence's last row: rows
// behind it come as zeros, and no tile needs a branch.
template <int D, bool V>
struct Stage {
  static constexpr int kPieces = D / 8;
  static constexpr int kPer = kTile * kPieces / 64 / kWaves;   // instructions of a wave
  int off[kPer];                            // bytes of this lane's pieces from the tile's first row
  const uint8_t* base;
  int64_t row_bytes;

  __device__ __forceinline__ void init(const void* p, int64_t stride, int wave, int lane) {
    base = reinterpret_cast<const uint8_t*>(p);
    row_bytes = 2 * stride;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = (wave * kPer + i) * 64 + lane, row = at / kPieces, slot = at % kPieces;
      off[i] = row * (int)row_bytes + 16 * (V ? v_piece<D>(row, slot) : k_piece<D>(row, slot));
    }
  }
  // keys [j0, j0 + kTile) of len
  __device__ __forceinline__ void start(int j0, int len, uint8_t* lds, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__               // (the host pass does not know descriptors)
    const int rows = min(len - j0, kTile);
    const int bytes = rows > 0 ? (rows - 1) * (int)row_bytes + 2 * D : 0;
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void*)(base + (rows > 0 ? j0 : 0) * row_bytes), 0, bytes, 0x00027000);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * kPer + i) * 1024),
                                               16, off[i], 0, 0, 0);
#endif
  }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 lds_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// A wave's state: 32 rows, row lane % 32.
template <typename T, int D>
struct Rows {
  u32x4 q[D / 16];
  f32x16 o[D / 32];
  float m, l;                               // reference, sum of the weights
  int last;                                 // last key the row sees, -1: none
};

// Scores of a tile.  With K as the first operand of a 32x32x16 product a lane
// gets 16 of 32 keys of one query row (column lane % 32): maximum and sum are
// nearly all inside a lane, and the weights are already the second operand
// of the product with V.
struct Scores {
  f32x16 s[2];                              // key 32 i + 8 (e / 4) + 4 hh + e % 4 in s[i][e]
};

template <typename T, int D>
__device__ __forceinline__ void scores(const Rows<T, D>& R, Scores& S, const uint8_t* kt, int lane) {
  const int col = lane & 31, hh = lane >> 5;
#pragma unroll
  for (int kb = 0; kb < D / 16; ++kb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 k = *reinterpret_cast<const u32x4*>(kt + ((32 * i + col) * (2 * D) + 16 * k_piece<D>(32 * i + col, 2 * kb + hh)));
      if (kb == 0)
        S.s[i] = T::mma32(k, R.q[kb], f32x16{});
      else
        S.s[i] = T::mma32(k, R.q[kb], S.s[i]);
    }
  }
}

// Weights of a tile's 64 keys, as operands: four groups of 16 keys.
struct Weights {
  u32x4 p[4];
};

// Scores as powers of two above the reference, in place; says whether some
// row's has to be raised, and gives the tile's largest.  (32-bit: an exponent is
// good to 2^-24 of how far apart score and reference are, as its score is to
// 2^-24 of itself.  Raising first, with exponents made once, costs 2.5%: 2048 rows
// behind 6144 keys 224 us, 229.)
// Masked, partly: some row of the workgroup does not see some key of the tile.
template <bool Masked, typename T, int D>
__device__ __forceinline__ bool exponents(const Rows<T, D>& R, Scores& S, float& mx, int j0, bool partly, float c,
                                          int lane) {
  const int hh = lane >> 5;
  const float base = R.m == kMinusInf ? 0.f : R.m;
#pragma unroll
  for (int e = 0; e < 32; ++e) S.s[e >> 4][e & 15] = __builtin_fmaf(S.s[e >> 4][e & 15], c, -base);
  if (Masked && partly) {
    const int seen = only_here(R.last - j0 - 4 * hh);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (32 * (e >> 4) + 8 * ((e & 15) >> 2) + (e & 3) > seen) S.s[e >> 4][e & 15] = kMinusInf;
  }
  float m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = fmaxf(fmaxf(S.s[i][0], S.s[i][1]), S.s[i][2]);
#pragma unroll
    for (int e = 3; e < 15; e += 2) m[i] = fmaxf(fmaxf(m[i], S.s[i][e]), S.s[i][e + 1]);
    m[i] = fmaxf(m[i], S.s[i][15]);
  }
  mx = max_halves(fmaxf(m[0], m[1]));
  return __any(mx > kMost || (R.m == kMinusInf && mx > kMinusInf));
}

template <typename T, int D>
__device__ __forceinline__ void raise_reference(Rows<T, D>& R, Scores& S, float mx) {
  const bool raise = mx > kMost || (R.m == kMinusInf && mx > kMinusInf);
  const float d = raise ? mx - kHead : 0.f;
  const float r = !raise ? 1.f : R.m == kMinusInf ? 0.f : exp2_fast(-d);
  if (raise) R.m = (R.m == kMinusInf ? 0.f : R.m) + d;
  R.l *= r;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) R.o[k] *= r;
#pragma unroll
  for (int e = 0; e < 32; ++e) S.s[e >> 4][e & 15] -= d;
}

template <typename T, int D>
__device__ __forceinline__ void weights(Rows<T, D>& R, const Scores& S, Weights& W) {
  float sum[4] = {R.l, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = exp2_fast(S.s[w >> 1][8 * (w & 1) + e]);
      sum[e & 3] += y[e];                   // (before they are rounded: the sum is an output)
    }
    W.p[w] = u32x4{T::cvt2(y[0], y[1]), T::cvt2(y[2], y[3]), T::cvt2(y[4], y[5]), T::cvt2(y[6], y[7])};
  }
  R.l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// The product with V, 32 columns x 16 keys an operand: transposing reads in
// the order of keys that the weights have.  (Addresses in one sum: the
// compiler follows a pointer to its buffer through few steps only, and waits
// for the copies under way where it does not know the buffer.)
template <int D>
__device__ __forceinline__ u32x4 value_operand(const uint8_t* vt, int k, int d, int lane) {
  // lane -> row (key) 4 hh + li / 4 of 16, 4 columns from 16 (gi & 1) + 4 (li % 4)
  const int li = lane & 15, gi = lane >> 4, hh = lane >> 5;
  const int row = 4 * hh + (li >> 2), vc = 2 * (gi & 1) + ((li & 3) >> 1), vb = 8 * (li & 1);
  // (the pieces' permutation goes by the row's last bits, the same for all k)
  const int at = row * (2 * D) + 16 * v_piece<D>(row, 4 * d + vc) + vb;
  const u32x2 a = lds_tr(vt + (at + 16 * k * (2 * D))), b = lds_tr(vt + (at + (16 * k + 8) * (2 * D)));
  return u32x4{a.x, a.y, b.x, b.y};
}

// In a masked tile a value that is not finite is kept out of the product
// (0 * inf would spoil rows that do not see its key) and given to the rows
// that see it at the end (add_special).
template <typename T>
__device__ __forceinline__ void take_special(u32x4& v) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t hi = (v[w] & (T::kExpOne << 16)) == (T::kExpOne << 16) ? 0xFFFF0000u : 0u;
    const uint32_t lo = (v[w] & T::kExpOne) == T::kExpOne ? 0xFFFFu : 0u;
    v[w] &= ~(hi | lo);
  }
}

// Says whether it met such values (Masked, partly as above; a sum of squares
// finds them, and very large ones).
template <bool Masked, typename T, int D>
__device__ __forceinline__ bool add_values(Rows<T, D>& R, const Weights& W, const uint8_t* vt, bool partly, int lane) {
  bool special = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u32x4 v[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) v[d] = value_operand<D>(vt, k, d, lane);
    if (Masked && partly) {
      float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int w = 0; w < 4; ++w) sq[w] = T::square2(v[d][w], sq[w]);
      if (__any(!((sq[0] + sq[1]) + (sq[2] + sq[3]) < __builtin_inff()))) {
        special = true;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) take_special<T>(v[d]);
      }
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d) R.o[d] = T::mma32(v[d], W.p[k], R.o[d]);
  }
  return special;
}

// Keys j0..j1-1 once more, for their values that are not finite.
template <typename T, int D>
__device__ void add_special(Rows<T, D>& R, const uint8_t* v, int64_t row_bytes, int j0, int j1, int lane) {
  const int hh = lane >> 5;
  for (int j = j0; j < j1; ++j) {
    const uint8_t* row = v + j * row_bytes + 8 * hh;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(row + 64 * d + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t bits = (i & 2 ? w.y : w.x) >> (16 * (i & 1)) & 0xFFFFu;
          const float x = (bits & T::kExpOne) == T::kExpOne ? T::lo(bits) : 0.f;
          if (j <= R.last) R.o[d][e + i] += x;
        }
      }
  }
}

template <int D>
struct Keys {
  Stage<D, false> k;
  Stage<D, true> v;
  int len;
};

// Step t: the scores of tile t and the weights of tile t-1 are there.  The
// product with tile t-1's V goes with the exponents of tile t, the scores of
// tile t+1 with the weights of tile t, so that the matrix core and the vector
// unit work at the same time in one wave too.  When every wave is through
// with step t-1, and the next K and the previous V have come, the copies of
// the next but one K and of this tile's V start; they have a whole step's
// time, and there is one barrier a step.  Tiles behind the last come as
// zeros, so only the scores ask which is the last (where tiles are masked: a
// short prompt's time is mostly one or two tiles').
template <bool First, bool Masked, typename T, int D>
__device__ __forceinline__ bool step(Rows<T, D>& R, Scores& S, Weights& W, const Keys<D>& K, int t,
                                     uint8_t* k_this, uint8_t* k_next, uint8_t* v_this, uint8_t* v_last, int n_whole,
                                     int t1, float c, int wave, int lane) {
  const int j0 = t * kTile;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  K.k.start(j0 + 2 * kTile, K.len, k_this, wave);
  if (!First) K.v.start(j0, K.len, v_this, wave);
  float mx;
  const bool raise = exponents<Masked, T, D>(R, S, mx, j0, t >= n_whole, c, lane);
  bool special = false;
  if (!First) special = add_values<Masked, T, D>(R, W, v_last, t > n_whole, lane);
  if (!First && !Masked) {
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {       // block A: D/8 products, 32 multiplications, 20 maxima
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, D == 64 ? 7 : 4, 0);
    }
  }
  if (raise) raise_reference<T, D>(R, S, mx);
  weights<T, D>(R, S, W);
  if (!Masked || t + 1 < t1) scores<T, D>(R, S, k_next, lane);
  // (the weights are made here, among the products, not where they are used)
#pragma unroll
  for (int w = 0; w < 4; ++w) asm volatile("" : "+v"(W.p[w]));
  asm volatile("" : "+v"(R.l));
  if (!Masked) {
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {       // block B: D/8 products, 32 exponentials, 32 additions, 16 conversions
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, D == 64 ? 10 : 5, 0);
    }
  }
  return special;
}

// Workgroup: 32*kWaves rows of one sequence and key head (row r = token
// r / group, query head r % group of the key head's group, so that the heads
// that share keys share the staged tiles), all keys they see, tile by tile
// in two LDS buffers: the next tile is on its way while one is computed.
//
// Bound by the card's power with heads of 128: 2048 rows behind 6144 keys, 32 + 8
// heads, 240 GFLOP in 224 us, 1.07 PFLOP/s; with zeros for inputs 161 us, since
// the clock falls to some 1.6 GHz under random ones (the library's largest
// product: 1.35 and 1.79 PFLOP/s).  With heads of 64 the vector unit does as
// much for half the products: 8 prompts of up to 2048, 32 + 4 heads, 104 us,
// 666 TFLOP/s, vector unit busy 61%, matrix core 33%.  A short prompt waits: one
// tile 6.0 us, each one more about 1 (2100 cycles for a wave alone on its SIMD,
// half of them the matrix core's).
// Weights are rounded once, to the row type: bf16 outputs are 0.0020 to 0.0023 of
// their size off, of which 0.0017 is their own rounding.  (What the rounding
// leaves as a second operand: 323 us for 224, 150 for 104; the largest score itself
// for a reference, at every tile, changes that by less than 0.0001 and takes 242
// and 114.)
// (64 rows a wave, one wave a SIMD: 278 and 154 us; 8 waves: 221 and 121; three
// buffers: 112 with heads of 64, and 309 rows, heads of 128, 12.9 for 12.2.)
template <typename T, int D>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : D > 64 ? 2 : 3) void prefill_kernel(PrefillArgs a, int tiles) {
  constexpr int kRowsWg = 32 * kWaves;
  constexpr int kBytes = kTile * D * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[kBytes], v0[kBytes], k1[kBytes], v1[kBytes];

  // (all arguments are asked for at once: fetched where they are used, each
  // line of them costs a short prompt a wait of its own)
  asm volatile("" ::"s"(a.cu_q), "s"(a.cu_k), "s"(a.B), "s"(a.Tq), "s"(a.Tk), "s"(a.max_q), "s"(a.per_q), "s"(a.per_k), "s"(a.Hq),
               "s"(a.Hk), "s"(a.q), "s"(a.k), "s"(a.v), "s"(a.out), "s"(a.lse), "s"(a.qs), "s"(a.ks), "s"(a.vs), "s"(a.os),
               "s"(a.c), "s"(a.causal), "s"(a.split.n));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go round robin over the 8 XCDs.  A key head's workgroups stay
  // on one of them, where its keys stay in the L2 (with fewer than 8 key heads
  // on 8/Hk of them, where 8/Hk is whole), so that each XCD has the
  // same share of every sequence.  The last rows, which see the most keys,
  // come first, those of all sequences.
  const int x = blockIdx.x & 7, b = (blockIdx.x >> 3) % a.B, i = (blockIdx.x >> 3) / a.B;
  int hk, qt;
  if (a.Hk % 8 == 0) {
    hk = x + 8 * (i % (a.Hk / 8));
    qt = tiles - 1 - i / (a.Hk / 8);
  } else {
    const int at = 8 * i + x;
    hk = at % a.Hk;
    qt = tiles - 1 - at / a.Hk;
  }
  if (qt < 0) return;                       // the whole workgroup
  const int group = a.Hq / a.Hk;
  const Seq sq = seq_rows(a.cu_q, a.per_q, a.Tq, b, a.q), sk = seq_rows(a.cu_k, a.per_k, a.Tk, b, a.q);
  const int rows = min(sq.n, a.max_q) * group, r0 = qt * kRowsWg;
  if (r0 >= rows) return;                   // the whole workgroup

  const int col = lane & 31, hh = lane >> 5;
  const int shift = sk.n - sq.n;            // key index of query row 0's own position
  Rows<T, D> R;
  const int r = r0 + wave * 32 + col;       // this lane's row
  const int token = r / group, h = hk * group + r % group;
  R.last = r >= rows ? -1 : a.causal ? min(shift + token, sk.n - 1) : sk.n - 1;
  R.m = kMinusInf;
  R.l = 0.f;
  {
    // (lanes behind the last row take it again: they see no key and write nothing)
    const int rc = min(r, rows - 1), hc = hk * group + rc % group;
    const uint16_t* p = (const uint16_t*)a.q + (int64_t)(sq.row0 + rc / group) * a.qs + (int64_t)hc * D + 8 * hh;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) R.q[k] = *reinterpret_cast<const u32x4*>(p + 16 * k);
  }
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) R.o[d][e] = 0.f;
  // tiles that all of the workgroup's rows see whole, and that any row sees
  const int last_row = min(r0 + kRowsWg, rows) - 1;
  const int all = a.causal ? min(shift + r0 / group, sk.n - 1) : sk.n - 1;
  const int any = a.causal ? shift + last_row / group : sk.n - 1;
  const int n_whole = all < 0 ? 0 : (all + 1) / kTile, n_tiles = any < 0 ? 0 : any / kTile + 1;

  // this part's tiles
  const int per = (n_tiles + a.split.n - 1) / a.split.n;
  const int t0 = blockIdx.y * per, t1 = min(t0 + per, n_tiles);

  if (t0 < t1) {
    Keys<D> K;
    K.len = sk.n;
    K.k.init((const uint16_t*)a.k + (int64_t)sk.row0 * a.ks + (int64_t)hk * D, a.ks, wave, lane);
    K.v.init((const uint16_t*)a.v + (int64_t)sk.row0 * a.vs + (int64_t)hk * D, a.vs, wave, lane);
    K.k.start(t0 * kTile, sk.n, k0, wave);
    K.k.start((t0 + 1) * kTile, sk.n, k1, wave);
    K.v.start(t0 * kTile, sk.n, v0, wave);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    Scores S;
    Weights W;
    scores<T, D>(R, S, k0, lane);
    step<true, true, T, D>(R, S, W, K, t0, k0, k1, v0, v1, n_whole, t1, a.c, wave, lane);
    int t = t0 + 1;
    const int t_whole = min(n_whole, t1);
    for (; t + 2 <= t_whole; t += 2) {
      step<false, false, T, D>(R, S, W, K, t, k1, k0, v1, v0, n_whole, t1, a.c, wave, lane);
      step<false, false, T, D>(R, S, W, K, t + 1, k0, k1, v0, v1, n_whole, t1, a.c, wave, lane);
    }
    const int masked_from = t - 1;          // (its V is still to come)
    bool special = false;
    for (; t < t1; t += 2) {
      special |= step<false, true, T, D>(R, S, W, K, t, k1, k0, v1, v0, n_whole, t1, a.c, wave, lane);
      if (t + 1 >= t1) break;
      special |= step<false, true, T, D>(R, S, W, K, t + 1, k0, k1, v0, v1, n_whole, t1, a.c, wave, lane);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    special |= add_values<true, T, D>(R, W, (t1 - t0) & 1 ? v0 : v1, t1 > n_whole, lane);
    if (special)
      add_special<T, D>(R, K.v.base, K.v.row_bytes, masked_from * kTile, min(t1 * kTile, sk.n), lane);
  }
  const float sum = sum_halves(R.l);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (r >= rows) return;
  const int64_t row = sq.row0 + token;
  if (a.split.n > 1) {
    const int64_t at = (blockIdx.y * (int64_t)a.Tq + row) * a.Hq + h;
    float* p = a.split.o + at * D + 4 * hh;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<f32x4*>(p + 32 * d + 2 * e) = f32x4{R.o[d][e], R.o[d][e + 1], R.o[d][e + 2], R.o[d][e + 3]};
    if (hh == 0) *reinterpret_cast<float2*>(a.split.ml + 2 * at) = make_float2(R.m, sum);
    return;
  }
  uint16_t* p = (uint16_t*)a.out + row * a.os + (int64_t)h * D + 4 * hh;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      u32x2 w;
      w.x = T::cvt2(R.o[d][e] * inv, R.o[d][e + 1] * inv);
      w.y = T::cvt2(R.o[d][e + 2] * inv, R.o[d][e + 3] * inv);
      *reinterpret_cast<u32x2*>(p + 32 * d + 2 * e) = w;
    }
  if (hh == 0 && a.lse) a.lse[row * a.Hq + h] = (R.m + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Joins the parts of one row and head: a wave each.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void join_parts_kernel(PrefillArgs a) {
  const int h = blockIdx.y * kWaves + (threadIdx.x >> 6), b = blockIdx.x / a.max_q, i = blockIdx.x % a.max_q;
  const Seq sq = seq_rows(a.cu_q, a.per_q, a.Tq, b, a.q);
  if (h >= a.Hq || i >= sq.n) return;
  const int64_t row = sq.row0 + i, at = row * a.Hq + h;
  join_row<T, D>(a.split.o + at * D, a.split.ml + 2 * at, a.split.n, (int64_t)a.Tq * a.Hq,
                 (uint16_t*)a.out + row * a.os + (int64_t)h * D, a.lse ? a.lse + at : nullptr, 1.f, threadIdx.x & 63);
}

template <typename T, int D>
hipError_t go(const PrefillArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hk);
  const int tiles = (int)((rows + 32 * kWaves - 1) / (32 * kWaves));
  const int64_t per_seq = ((int64_t)tiles * a.Hk + 7) / 8 * 8;   // whole rounds of the XCDs
  hipLaunchKernelGGL((prefill_kernel<T, D>), dim3((unsigned)(per_seq * a.B), (unsigned)a.split.n), dim3(kThreads), 0, s, a, tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.split.n == 1) return e;
  hipLaunchKernelGGL((join_parts_kernel<T, D>), dim3((unsigned)((int64_t)a.B * a.max_q), (unsigned)((a.Hq + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t by_dim(const PrefillArgs& a, hipStream_t s) {
  switch (a.D) {
    case 64: return go<T, 64>(a, s);
    case 128: return go<T, 128>(a, s);
    default: return go<T, 256>(a, s);
  }
}

}  // namespace

namespace qmoe {

// Parts the keys are cut into where the rows alone would leave much of the
// card idle: up to 4/3 workgroups a compute unit, each with 8 tiles of the
// average context at least (fewer do not pay for the join).
int attn_prefill_parts(const PrefillArgs& a, int cus) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hk);
  const int64_t wgs = (rows + 32 * kWaves - 1) / (32 * kWaves) * a.B * a.Hk;
  const int64_t most = a.Tk / a.B / (8 * kTile);
  int64_t n = 4ll * cus / 3 / wgs;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

hipError_t launch_attn_prefill(const PrefillArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? by_dim<Bf16>(a, s) : by_dim<F16>(a, s);
}

}  // namespace qmoe

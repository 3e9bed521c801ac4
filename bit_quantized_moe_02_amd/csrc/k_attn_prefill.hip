// Attention of packed prompts (moe_attn_prefill).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_common.hpp"

using namespace qmoe;
using namespace qmoe_dev;

namespace {

constexpr int kTile = 64;                   // keys a workgroup stages at once
constexpr int kWaves = 4;
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

// Starts the copy of keys [j0, j0 + kTile) (rows behind the last repeat it)
// into LDS: 1024 bytes an instruction, which go there in lane order.
template <int D, bool V>
__device__ __forceinline__ void stage(const uint16_t* base, int64_t stride, int j0, int len, uint8_t* lds, int wave,
                                      int lane) {
  constexpr int kPieces = D / 8;
  constexpr int kPer = kTile * kPieces / 64 / kWaves;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = (wave * kPer + i) * 64 + lane;
    const int row = at / kPieces, slot = at % kPieces;
    const int piece = V ? v_piece<D>(row, slot) : k_piece<D>(row, slot);
    const uint16_t* src = base + (int64_t)min(j0 + row, len - 1) * stride + 8 * piece;
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)(lds + (wave * kPer + i) * 1024), 16, 0, 0);
  }
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 lds_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// A wave's state: 32*CT rows, row lane % 32 of each group of 32.
template <typename T, int D, int CT>
struct Rows {
  u32x4 q[CT][D / 16];
  f32x16 o[CT][D / 32];
  float m[CT], l[CT];
  int last[CT];                             // last key the row sees, -1: none
};

// One tile of keys.  With K as the first operand of a 32x32x16 product a
// lane gets 16 of 32 keys of one query row (column lane % 32): maximum and
// sum are nearly all inside a lane, and the weights are already the second
// operand of the product with V, whose first operand (columns x keys) comes
// out of LDS by transposing reads in the same order of keys.
template <typename T, int D, int CT>
__device__ __forceinline__ void tile_step(Rows<T, D, CT>& R, const uint8_t* kt, const uint8_t* vt, int j0, bool all,
                                          float c, int lane) {
  const int col = lane & 31, hh = lane >> 5;
  f32x16 s[CT][2];
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[t][i][e] = 0.f;
#pragma unroll
  for (int kb = 0; kb < D / 16; ++kb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 k = *reinterpret_cast<const u32x4*>(kt + (32 * i + col) * (2 * D) + 16 * k_piece<D>(32 * i + col, 2 * kb + hh));
#pragma unroll
      for (int t = 0; t < CT; ++t) s[t][i] = T::mma32(k, R.q[t][kb], s[t][i]);
    }
  }
  if (!all) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (j0 + 32 * i + 8 * (e >> 2) + 4 * hh + (e & 3) > R.last[t]) s[t][i][e] = kMinusInf;
  }
  u32x4 p[CT][4];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    float mx = kMinusInf;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 2) mx = fmaxf(mx, fmaxf(s[t][i][e], s[t][i][e + 1]));
    mx = max_halves(mx) * c;
    if (__any(mx > R.m[t])) {
      mx = fmaxf(R.m[t], mx);
      const float r = R.m[t] == kMinusInf ? 0.f : exp2_fast(R.m[t] - mx);
      R.l[t] *= r;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) R.o[t][d] *= r;
      R.m[t] = mx;
    }
    const float base = R.m[t] == kMinusInf ? 0.f : R.m[t];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[t][i][e] = exp2_fast(__builtin_fmaf(s[t][i][e], c, -base));
        R.l[t] += s[t][i][e];
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        u32x4 x;
        x.x = T::cvt2(s[t][i][8 * w], s[t][i][8 * w + 1]);
        x.y = T::cvt2(s[t][i][8 * w + 2], s[t][i][8 * w + 3]);
        x.z = T::cvt2(s[t][i][8 * w + 4], s[t][i][8 * w + 5]);
        x.w = T::cvt2(s[t][i][8 * w + 6], s[t][i][8 * w + 7]);
        p[t][2 * i + w] = x;
      }
    }
  }
  // V: lane -> row (key) 4 hh + li / 4 of 16, 4 columns from 16 (gi & 1) + 4 (li % 4)
  const int li = lane & 15, gi = lane >> 4;
  const int row = 4 * hh + (li >> 2), vc = 2 * (gi & 1) + ((li & 3) >> 1), vb = 8 * (li & 1);
  uint32_t special = 0;                     // exponents of all ones among V's values
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const int ra = 16 * k + row, rb = ra + 8;
      const u32x2 a = lds_tr(vt + ra * (2 * D) + 16 * v_piece<D>(ra, 4 * d + vc) + vb);
      const u32x2 b = lds_tr(vt + rb * (2 * D) + 16 * v_piece<D>(rb, 4 * d + vc) + vb);
      u32x4 v = {a.x, a.y, b.x, b.y};
      if (!all) {
        // a value that is not finite is kept out of the product (0 * inf
        // would spoil rows that do not see its key) and given below
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t hi = (v[w] & (T::kExpOne << 16)) == (T::kExpOne << 16) ? 0xFFFF0000u : 0u;
          const uint32_t lo = (v[w] & T::kExpOne) == T::kExpOne ? 0xFFFFu : 0u;
          special |= hi | lo;
          v[w] &= ~(hi | lo);
        }
      }
#pragma unroll
      for (int t = 0; t < CT; ++t) R.o[t][d] = T::mma32(v, p[t][k], R.o[t][d]);
    }
  }
  if (!all && __any(special != 0)) {
    for (int j = 0; j < kTile; ++j) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int cc = 32 * d + 8 * (e >> 2) + 4 * hh + (e & 3);
          const uint32_t bits = *reinterpret_cast<const uint16_t*>(vt + j * (2 * D) + 16 * v_piece<D>(j, cc >> 3) + 2 * (cc & 7));
          if ((bits & T::kExpOne) != T::kExpOne) continue;
#pragma unroll
          for (int t = 0; t < CT; ++t)
            if (j0 + j <= R.last[t]) R.o[t][d][e] += T::lo(bits);
        }
    }
  }
}

// Workgroup: 32*CT*kWaves rows of one sequence and key head (row r = token
// r / group, query head r % group of the key head's group, so that the heads
// that share keys share the staged tiles), all keys they see, tile by tile
// in two LDS buffers: the next tile is on its way while one is computed.
template <typename T, int D, int CT>
__global__ __launch_bounds__(kThreads, CT == 1 && D <= 128 ? 2 : 1) void prefill_kernel(PrefillArgs a, int tiles) {
  constexpr int kRowsWg = 32 * CT * kWaves;
  constexpr int kBytes = kTile * D * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[kBytes], v0[kBytes], k1[kBytes], v1[kBytes];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = a.B * a.Hk;
  // the longest rows first; workgroups of one key head on one XCD (workgroups
  // go round robin over the 8), where their keys stay in its L2
  int pair, qt;
  if (pairs % 8 == 0) {
    const int x = blockIdx.x & 7, i = blockIdx.x >> 3;
    pair = x + 8 * (i / tiles);
    qt = tiles - 1 - i % tiles;
  } else {
    pair = blockIdx.x % pairs;
    qt = tiles - 1 - blockIdx.x / pairs;
  }
  const int b = pair / a.Hk, hk = pair % a.Hk;
  const int group = a.Hq / a.Hk;
  const Seq sq = seq_rows(a.cu_q, a.per_q, a.Tq, b), sk = seq_rows(a.cu_k, a.per_k, a.Tk, b);
  const int rows = sq.n * group, r0 = qt * kRowsWg;
  if (r0 >= rows) return;                   // the whole workgroup

  const int col = lane & 31, hh = lane >> 5;
  const int shift = sk.n - sq.n;            // key index of query row 0's own position
  const int w0 = r0 + wave * 32 * CT;       // this wave's first row
  Rows<T, D, CT> R;
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int r = w0 + 32 * t + col;
    const int i = r / group, h = hk * group + r % group;
    R.last[t] = r >= rows ? -1 : a.causal ? min(shift + i, sk.n - 1) : sk.n - 1;
    R.m[t] = kMinusInf;
    R.l[t] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) R.q[t][k] = u32x4{0, 0, 0, 0};
    if (r < rows) {
      const uint16_t* p = (const uint16_t*)a.q + (int64_t)(sq.row0 + i) * a.qs + (int64_t)h * D + 8 * hh;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) R.q[t][k] = *reinterpret_cast<const u32x4*>(p + 16 * k);
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) R.o[t][d][e] = 0.f;
  }
  // keys that all rows of the wave see, and that any does
  const int w_end = min(w0 + 32 * CT, rows) - 1, wg_end = min(r0 + kRowsWg, rows) - 1;
  const int w_all = a.causal ? min(shift + w0 / group, sk.n - 1) : sk.n - 1;
  const int w_any = w0 >= rows ? -1 : a.causal ? shift + w_end / group : sk.n - 1;
  const int wg_any = a.causal ? shift + wg_end / group : sk.n - 1;
  const int n_tiles = wg_any < 0 || sk.n == 0 ? 0 : wg_any / kTile + 1;

  const uint16_t* kbase = (const uint16_t*)a.k + (int64_t)sk.row0 * a.ks + (int64_t)hk * D;
  const uint16_t* vbase = (const uint16_t*)a.v + (int64_t)sk.row0 * a.vs + (int64_t)hk * D;
  if (n_tiles > 0) {
    stage<D, false>(kbase, a.ks, 0, sk.n, k0, wave, lane);
    stage<D, true>(vbase, a.vs, 0, sk.n, v0, wave, lane);
  }
  for (int t = 0; t < n_tiles; t += 2) {
    // this tile has come, for every wave; and every wave is done with the
    // other buffer, which the next tile may now fill
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t + 1 < n_tiles) {
      stage<D, false>(kbase, a.ks, (t + 1) * kTile, sk.n, k1, wave, lane);
      stage<D, true>(vbase, a.vs, (t + 1) * kTile, sk.n, v1, wave, lane);
    }
    if (t * kTile <= w_any) tile_step<T, D, CT>(R, k0, v0, t * kTile, t * kTile + kTile - 1 <= w_all, a.c, lane);
    if (t + 1 >= n_tiles) break;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t + 2 < n_tiles) {
      stage<D, false>(kbase, a.ks, (t + 2) * kTile, sk.n, k0, wave, lane);
      stage<D, true>(vbase, a.vs, (t + 2) * kTile, sk.n, v0, wave, lane);
    }
    if ((t + 1) * kTile <= w_any)
      tile_step<T, D, CT>(R, k1, v1, (t + 1) * kTile, (t + 1) * kTile + kTile - 1 <= w_all, a.c, lane);
  }
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const float sum = sum_halves(R.l[t]);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int r = w0 + 32 * t + col;
    if (r >= rows) continue;
    const int tok = sq.row0 + r / group, h = hk * group + r % group;
    uint16_t* p = (uint16_t*)a.out + (int64_t)tok * a.os + (int64_t)h * D + 4 * hh;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        u32x2 w;
        w.x = T::cvt2(R.o[t][d][e] * inv, R.o[t][d][e + 1] * inv);
        w.y = T::cvt2(R.o[t][d][e + 2] * inv, R.o[t][d][e + 3] * inv);
        *reinterpret_cast<u32x2*>(p + 32 * d + 2 * e) = w;
      }
    if (hh == 0 && a.lse) a.lse[(int64_t)tok * a.Hq + h] = (R.m[t] + __builtin_amdgcn_logf(sum)) * kLn2;
  }
}

template <typename T, int D, int CT>
hipError_t go(const PrefillArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hk);
  const int tiles = (int)((rows + 32 * CT * kWaves - 1) / (32 * CT * kWaves));
  hipLaunchKernelGGL((prefill_kernel<T, D, CT>), dim3((unsigned)((int64_t)tiles * a.B * a.Hk)), dim3(kThreads), 0, s,
                     a, tiles);
  return hipGetLastError();
}

template <typename T>
hipError_t by_dim(const PrefillArgs& a, hipStream_t s) {
  switch (a.D) {
    case 64: return go<T, 64, 1>(a, s);
    case 128: return go<T, 128, 1>(a, s);
    default: return go<T, 256, 1>(a, s);
  }
}

}  // namespace

namespace qmoe {

hipError_t launch_attn_prefill(const PrefillArgs& a, int dtype, int cus, hipStream_t s) {
  (void)cus;
  return dtype == 0 ? by_dim<Bf16>(a, s) : by_dim<F16>(a, s);
}

}  // namespace qmoe

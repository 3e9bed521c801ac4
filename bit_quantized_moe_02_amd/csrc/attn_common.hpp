// Device helpers shared by the attention kernels: row types, the 8-bit cache
// (layout in include/qmoe_attn.h), sequences of a step.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "k_attn.h"

namespace qmoe_dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kMinusInf = -__builtin_inff();
constexpr float kLn2 = 0.6931471805599453f;

// The two row types.  cvt2 packs two values rounded to nearest even; dec2
// makes two codes (bytes 0,1 or 2,3 of w) times the power of two `scale`
// into two values, exact unless they leave the type's range.
struct Bf16 {
  typedef bf16x8 v8;
  static __device__ __forceinline__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t cvt2(float a, float b) {
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ uint32_t dec2(uint32_t w, float scale, bool upper) {
    return upper ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))
                 : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
  }
  static __device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma32(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kExpOne = 0x7F80u;
  static constexpr int kOver = 120;         // codes times 2^kOver may leave the type's range
  // acc + lo^2 + hi^2
  static __device__ __forceinline__ float square2(uint32_t w, float acc) {
    const bf16x2 v = __builtin_bit_cast(bf16x2, w);
    return __builtin_amdgcn_fdot2_f32_bf16(v, v, acc, false);
  }
};

struct F16 {
  typedef f16x8 v8;
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).x; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).y; }
  static __device__ __forceinline__ uint32_t cvt2(float a, float b) {
    const f16x2 r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ uint32_t dec2(uint32_t w, float scale, bool upper) {
    return upper ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true))
                 : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false));
  }
  static __device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma32(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t kExpOne = 0x7C00u;
  static constexpr int kOver = 8;
  static __device__ __forceinline__ float square2(uint32_t w, float acc) {
    const f16x2 v = __builtin_bit_cast(f16x2, w);
    return __builtin_amdgcn_fdot2(v, v, acc, false);
  }
};

// Eight codes (two words) times a power of two: an MFMA operand.
template <typename T>
__device__ __forceinline__ u32x4 dec8(uint32_t w0, uint32_t w1, float scale) {
  u32x4 r;
  r.x = T::dec2(w0, scale, false);
  r.y = T::dec2(w0, scale, true);
  r.z = T::dec2(w1, scale, false);
  r.w = T::dec2(w1, scale, true);
  return r;
}

// A sequence of a step: its length, its n rows and the first of them; row i
// is position len - n + i.
struct Seq {
  int len, n, row0;
};

// `some`: an address of 8 bytes that may be read, for where there is no cu (no
// branch then keeps this load from going with others).
__device__ __forceinline__ Seq seq_rows(const int32_t* cu, int per_seq, int T, int b, const void* some) {
  const int32_t* p = cu ? cu + b : (const int32_t*)some;
  const int first = p[0], past = p[1];
  const int c0 = min(max(first, 0), T), c1 = min(max(past, c0), T);
  Seq s;
  s.len = 0;
  s.row0 = cu ? c0 : b * per_seq;
  s.n = cu ? c1 - c0 : per_seq;
  return s;
}

__device__ __forceinline__ Seq seq_of(const qmoe::KvArgs& a, int b) {
  const int len = a.lens[b];
  Seq s = seq_rows(a.cu, a.per_seq, a.T, b, a.codes);
  s.len = min(max(len, 0), a.max_len);
  return s;
}

// Index of block `blk` of sequence b and head hk in the cache, -1 when its
// page is none of the cache's.  blk must lie inside the page table.
__device__ __forceinline__ int64_t block_of(const qmoe::KvArgs& a, int b, int blk, int hk) {
  const int page = a.table[(int64_t)b * a.table_stride + (blk >> a.lb)];
  if ((unsigned)page >= (unsigned)a.n_pages) return -1;
  return ((((int64_t)page * a.Hk + hk) << a.lb) + (blk & ((1 << a.lb) - 1)));
}

// Maximum over the four 16-lane rows of a wave (same lane of each): every
// lane gets it.
__device__ __forceinline__ float max_rows4(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  const float y = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  const auto c = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, y),
                                                  false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)c[0]), __builtin_bit_cast(float, (uint32_t)c[1]));
}

__device__ __forceinline__ float sum_rows4(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  const float y = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  const auto c = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, y),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)c[0]) + __builtin_bit_cast(float, (uint32_t)c[1]);
}

// Maximum and sum over the two halves of a wave (lane and lane + 32).
__device__ __forceinline__ float max_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
}

__device__ __forceinline__ float sum_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// One wave joins the n parts of one row and head, 4 columns a lane, as many
// parts at once as it has lanes for: part p's un-normalised output at
// o + p * pitch * D (1 / up times its size), its (maximum, sum) at ml + 2 * p *
// pitch; lse may be null.
template <typename T, int D>
__device__ __forceinline__ void join_row(const float* o, const float* ml, int n, int64_t pitch, uint16_t* out, float* lse,
                                         float up, int lane) {
  constexpr int kCh = D / 4, kAtOnce = 64 / kCh;
  const int ch = lane % kCh, p0 = lane / kCh;
  float mx = kMinusInf;
  for (int p = lane; p < n; p += 64) mx = fmaxf(mx, ml[2 * p * pitch]);
  for (int s = 32; s >= 1; s >>= 1) mx = fmaxf(mx, __shfl_xor(mx, s));
  const float base = mx == kMinusInf ? 0.f : mx;
  float sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = p0; p < n; p += kAtOnce) {
    const float2 v = *reinterpret_cast<const float2*>(ml + 2 * p * pitch);
    const float e = exp2_fast(v.x - base);  // (a part that saw nothing: maximum -inf, zeros)
    sum += e * v.y;
    acc += *reinterpret_cast<const f32x4*>(o + p * pitch * D + 4 * ch) * e;
  }
#pragma unroll
  for (int s = kCh; s < 64; s <<= 1) {
    sum += __shfl_xor(sum, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], s);
  }
  if (p0 != 0) return;
  const float inv = sum == 0.f ? 0.f : up / sum;
  u32x2 w;
  w.x = T::cvt2(acc[0] * inv, acc[1] * inv);
  w.y = T::cvt2(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<u32x2*>(out + 4 * ch) = w;
  if (ch == 0 && lse) *lse = (mx + __builtin_amdgcn_logf(sum)) * kLn2;
}

}  // namespace qmoe_dev

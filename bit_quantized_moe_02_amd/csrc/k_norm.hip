// Root-mean-square norm with the residual's addition (moe_rms_norm).
//
//   h = x + residual, rounded to the residual's type;  y = h / sqrt(mean(h^2) + eps) * weight
//
// Bytes bound it: each value is read and written once, a vector staying in
// registers, 8 columns a thread and pass, between the sum of its squares and the
// outputs.  The sum of squares is held in 64 bits, and where y becomes 8-bit codes so is y:
// a code next to the border of two, or on it, is then the one of the formula.  In 64 bits that is some 10 operations a
// value, 2 to 5 % of the time of many vectors and 0.5 us of a few long ones'.
//
// Vectors of up to 512 columns take the least power of two of lanes that holds
// them (several to a wave, no barrier); longer ones a workgroup of 8 columns a
// thread, up to 1024 threads, then two passes of that.  Half the threads with twice
// the passes were slower for 4096 columns (1 row 3.7 for 3.2 us) and 16384 (8192 rows 239
// for 227) and no faster for 7168.  Lanes add up by moves between registers; through LDS'
// exchange the same sums cost 0.2 to 0.5 us a call.
//
// bf16, sum and outputs: 4096 rows of 7168 columns to bf16 45 us (5.2 TB/s), to codes
// 43 (4.8), to both 52; 8192 of 16384 to codes 214 (4.4).  One row of 512 2.1 us (an empty kernel
// 2.0), of 7168 3.0, as codes 3.8; 64 rows of 7168 as codes 4.3.  Heads of 128 without a sum: 48 of
// one token 2.5 us, of 64 2.7, of 8192 40 (5.1 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmoe_step.h"
#include "k_step.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int T>
struct Raw {                       // 8 values of a type
  u32x4 v[T == MOE_DT_F32 ? 2 : 1];
};

template <int T>
__device__ __forceinline__ Raw<T> load8(const void* p, int64_t at) {
  Raw<T> r;
  if (T == MOE_DT_F32) {
    const u32x4* q = (const u32x4*)((const float*)p + at);
    r.v[0] = q[0];
    r.v[T == MOE_DT_F32] = q[1];
  } else {
    r.v[0] = *(const u32x4*)((const uint16_t*)p + at);
  }
  return r;
}

template <int T>
__device__ __forceinline__ void to_f32(const Raw<T>& r, float* f) {
  for (int i = 0; i < 8; ++i) {
    const uint32_t word = r.v[T == MOE_DT_F32 ? i / 4 : 0][i % 4];    // (a bit cast takes a copy: of a vector's element it reads the first)
    if (T == MOE_DT_F32) f[i] = __builtin_bit_cast(float, word);
    else if (T == MOE_DT_BF16) f[i] = __builtin_bit_cast(float, i % 2 ? r.v[0][i / 2] & 0xFFFF0000u : r.v[0][i / 2] << 16);
    else f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.v[0][i / 2] >> (16 * (i % 2))));
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, bf2));
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, h2));
}

template <int T>
__device__ __forceinline__ Raw<T> from_f32(const float* f) {
  Raw<T> r;
  if (T == MOE_DT_F32) {
    for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = __builtin_bit_cast(uint32_t, f[i]);
  } else {
    for (int i = 0; i < 4; ++i)
      r.v[0][i] = T == MOE_DT_BF16 ? bf16_pair(f[2 * i], f[2 * i + 1]) : f16_pair(f[2 * i], f[2 * i + 1]);
  }
  return r;
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t at, const Raw<T>& r) {
  if (T == MOE_DT_F32) {
    u32x4* q = (u32x4*)((float*)p + at);
    q[0] = r.v[0];
    q[1] = r.v[T == MOE_DT_F32];
  } else {
    *(u32x4*)((uint16_t*)p + at) = r.v[0];
  }
}

__device__ __forceinline__ void store8_as(int type, void* p, int64_t at, const float* f) {
  if (type == MOE_DT_F32) store8<MOE_DT_F32>(p, at, from_f32<MOE_DT_F32>(f));
  else if (type == MOE_DT_BF16) store8<MOE_DT_BF16>(p, at, from_f32<MOE_DT_BF16>(f));
  else store8<MOE_DT_F16>(p, at, from_f32<MOE_DT_F16>(f));
}

__device__ __forceinline__ void weight8(const NormArgs& a, int col, float* f) {
  if (!a.w) {
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  } else if (a.wt == MOE_DT_F32) {
    to_f32<MOE_DT_F32>(load8<MOE_DT_F32>(a.w, col), f);
  } else if (a.wt == MOE_DT_BF16) {
    to_f32<MOE_DT_BF16>(load8<MOE_DT_BF16>(a.w, col), f);
  } else {
    to_f32<MOE_DT_F16>(load8<MOE_DT_F16>(a.w, col), f);
  }
}

// For codes, a quotient q of less than 2^19 gets 1.5 * 2^20 + 1/2 + 2^-31 added: the upper word of the sum is the whole
// number next to q, above kZero, and the lower one, q's distance above the half between two codes, is at most kBorder where
// q is within 2^-31 of a half.
constexpr double kToCode = 1572864.5 + 0x1p-31;
constexpr int kZero = 0x41380000;
constexpr uint32_t kBorder = 4;

// |y| as an unsigned number, which orders as |y| does, not a number on top.
__device__ __forceinline__ uint32_t size_bits(float y) { return __builtin_bit_cast(uint32_t, y) & 0x7FFFFFFFu; }

// The value of the lane d away (d < 16; of lanes that hold the same values in each d).
template <int D>
__device__ __forceinline__ uint32_t beside(uint32_t v) {
  constexpr int kMove = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;   // within four lanes, mirrored within 8, within 16
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kMove, 0xF, 0xF, true);
}
template <int D>
__device__ __forceinline__ double beside(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const uint32_t lo = b[0], hi = b[1];
  return __builtin_bit_cast(double, (u32x2){beside<D>(lo), beside<D>(hi)});
}
// Both values of lanes d away (16: next rows of 16; 32: the halves of the wave), the same two in both.
template <int D>
__device__ __forceinline__ u32x2 both(uint32_t v) {
  return __builtin_bit_cast(u32x2, D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false) : __builtin_amdgcn_permlane32_swap(v, v, false, false));
}
template <int LANES>
__device__ __forceinline__ double sum_of(double v) {   // of LANES neighbours, to each
  if constexpr (LANES >= 2) v += beside<1>(v);
  if constexpr (LANES >= 4) v += beside<2>(v);
  if constexpr (LANES >= 8) v += beside<4>(v);
  if constexpr (LANES >= 16) v += beside<8>(v);
  if constexpr (LANES >= 32) {
    const u32x2 b = __builtin_bit_cast(u32x2, v);
    const uint32_t lo = b[0], hi = b[1];
    const u32x2 l = both<16>(lo), h = both<16>(hi);
    v = __builtin_bit_cast(double, (u32x2){l[0], h[0]}) + __builtin_bit_cast(double, (u32x2){l[1], h[1]});
  }
  if constexpr (LANES >= 64) {
    const u32x2 b = __builtin_bit_cast(u32x2, v);
    const uint32_t lo = b[0], hi = b[1];
    const u32x2 l = both<32>(lo), h = both<32>(hi);
    v = __builtin_bit_cast(double, (u32x2){l[0], h[0]}) + __builtin_bit_cast(double, (u32x2){l[1], h[1]});
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  if constexpr (LANES >= 2) v = max(v, beside<1>(v));
  if constexpr (LANES >= 4) v = max(v, beside<2>(v));
  if constexpr (LANES >= 8) v = max(v, beside<4>(v));
  if constexpr (LANES >= 16) v = max(v, beside<8>(v));
  if constexpr (LANES >= 32) {
    const u32x2 b = both<16>(v);
    v = max(b[0], b[1]);
  }
  if constexpr (LANES >= 64) {
    const u32x2 b = both<32>(v);
    v = max(b[0], b[1]);
  }
  return v;
}

constexpr int kResNone = -1;

// LANES <= 64: that many lanes of a wave take a vector, without LDS; more: a workgroup of
// LANES threads takes one.  A thread holds 8 columns of each pass of 8 * LANES.
template <int XT, int RT, int LANES, int PASSES>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES) void norm_kernel(NormArgs a) {
  constexpr bool kWave = LANES <= 64;
  constexpr int kWaves = kWave ? 1 : LANES / 64;
  __shared__ double part[kWave ? 1 : kWaves];
  __shared__ uint32_t top[kWave ? 1 : kWaves];
  const int lane = kWave ? threadIdx.x % LANES : threadIdx.x;
  // (below 2^24 vectors)
  const uint32_t vec = kWave ? blockIdx.x * (256 / LANES) + threadIdx.x / LANES : blockIdx.x;
  const bool here = vec < (uint32_t)a.rows * (uint32_t)a.heads;
  const int row = !here ? 0 : a.heads == 1 ? vec : vec / (uint32_t)a.heads, head = here ? vec - (uint32_t)row * a.heads : 0;
  const int64_t first = (int64_t)head * a.cols;
  const int64_t xat = row * a.xs + first, rat = row * a.rs + first;

  constexpr int RTx = RT == kResNone ? XT : RT;
  Raw<XT> x[PASSES];
  Raw<RTx> r[PASSES];
  float h[PASSES][8], w[PASSES][8];
  bool in[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int col = (p * LANES + lane) * 8;
    in[p] = here && col < a.cols;
    if (in[p]) {
      x[p] = load8<XT>(a.x, xat + col);
      if (RT != kResNone) r[p] = load8<RTx>(a.res, rat + col);
    }
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
    if (in[p]) weight8(a, (p * LANES + lane) * 8, w[p]);
  double ss = 0;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if (in[p]) {
      to_f32<XT>(x[p], h[p]);
      if (RT != kResNone) {
        float f[8];
        to_f32<RTx>(r[p], f);
        for (int i = 0; i < 8; ++i) h[p][i] += f[i];
        const Raw<RTx> s = from_f32<RTx>(h[p]);        // (the norm is of the sum as it is kept)
        to_f32<RTx>(s, h[p]);
        if (a.sum) store8<RTx>(a.sum, row * a.ss + first + (p * LANES + lane) * 8, s);
      }
    } else {
      for (int i = 0; i < 8; ++i) h[p][i] = 0, w[p][i] = 0;
    }
    for (int i = 0; i < 8; ++i) ss = fma((double)h[p][i], (double)h[p][i], ss);
  }
  if (!a.out && !a.codes) return;
  ss = sum_of<kWave ? LANES : 64>(ss);
  if (!kWave) {
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = ss;
    __syncthreads();
    ss = sum_of<kWaves>(part[threadIdx.x % kWaves]);
  }
  const double inv = rsqrt(ss * a.per_col + (double)a.eps);

  if (a.out) {
    const float f = (float)inv;
    // A 32-bit root holds its 24 bits, and is finite, for all but values near the largest (of a mean square above 2^252) and,
    // without epsilon, the smallest numbers: there in 64 bits.
    const bool holds = f >= 0x1p-126f && f <= 0x1p127f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!in[p]) continue;
      float y[8];
      for (int i = 0; i < 8; ++i) y[i] = h[p][i] * f * w[p][i];
      if (!holds)
        for (int i = 0; i < 8; ++i) y[i] = (float)((double)h[p][i] * inv * (double)w[p][i]);
      store8_as(a.ot, a.out, row * a.os + first + (p * LANES + lane) * 8, y);
    }
  }
  if (!a.codes) return;

  // 8 bits: y in 64 bits, its sizes compared as 32-bit numbers (rounding keeps their order)
  uint32_t m[PASSES];
  uint32_t all = 0;
  double y[PASSES][8];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    m[p] = 0;
    for (int i = 0; i < 8; ++i) {
      y[p][i] = (double)h[p][i] * inv * (double)w[p][i];
      m[p] = max(m[p], size_bits((float)y[p][i]));
    }
    all = max(all, m[p]);
  }
  const int groups = a.group ? (a.cols + a.group - 1) / a.group : 1;
  if (a.group) {                                       // 128 columns: 16 lanes
#pragma unroll
    for (int p = 0; p < PASSES; ++p) m[p] = max_of<LANES < 16 ? LANES : 16>(m[p]);
  } else {
    all = max_of<kWave ? LANES : 64>(all);
    if (!kWave) {
      if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = all;
      __syncthreads();
      all = max_of<kWaves>(top[threadIdx.x % kWaves]);
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) m[p] = all;
  }
  u32x2 c[PASSES];
  float scale[PASSES];
  uint32_t border = ~0u;
  auto put = [&](u32x2& c, int i, int q) {
    c[i / 4] |= ((uint32_t)min(max(q, kZero - 127), kZero + 127) & 0xFFu) << (8 * (i % 4));
  };
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const bool fine = m[p] < 0x7F800000u;
    scale[p] = fine ? __builtin_bit_cast(float, m[p]) / 127.0f : __builtin_nanf("");
    const double back = fine && scale[p] > 0 ? 1.0 / (double)scale[p] : 0.0;
    c[p] = (u32x2){0, 0};
    uint32_t next = ~0u;
    for (int i = 0; i < 8; ++i) {
      // (scales below the normal numbers are so much rounded that codes can pass 127, to 190 at most)
      const uint64_t at = __builtin_bit_cast(uint64_t, fma(y[p][i], back, kToCode));
      put(c[p], i, (int)(at >> 32));
      next = min(next, (uint32_t)at);
    }
    if (back == 0.0) c[p] = (u32x2){0, 0};                // (products that may be not a number)
    else border = min(border, next);
  }
  if (border <= kBorder) {
    // The products by reciprocals are within 2^-42 of y / scale, so that only here a code may be on the other side of a
    // half, or on one: the formula's own divisions, of which one value in 2^29 has need.
    const double root = sqrt(ss / a.cols + (double)a.eps);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!(scale[p] > 0)) continue;
      c[p] = (u32x2){0, 0};
      for (int i = 0; i < 8; ++i) {
        float hv = h[p][i], wv = w[p][i];
        asm("" : "+v"(hv), "+v"(wv));                     // (their 64-bit forms made anew, not kept: registers)
        put(c[p], i, kZero + (int)rint((double)hv / root * (double)wv / (double)scale[p]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if (!in[p]) continue;
    const int col = (p * LANES + lane) * 8;
    *(u32x2*)(a.codes + row * a.cs + first + col) = c[p];
    const int g = a.group ? col / a.group : 0;
    if (col == g * (a.group ? a.group : 1)) a.scales[((int64_t)head * groups + g) * a.scs + row] = scale[p];
  }
}

template <int XT, int RT>
hipError_t launch_types(const NormArgs& a, hipStream_t s) {
  const int64_t n = (int64_t)a.rows * a.heads;
#define WAVE(L) norm_kernel<XT, RT, L, 1><<<dim3((unsigned)((n + 256 / L - 1) / (256 / L))), dim3(256), 0, s>>>(a)
#define GROUP(L, P) norm_kernel<XT, RT, L, P><<<dim3((unsigned)n), dim3(L), 0, s>>>(a)
  switch (norm_threads(a.cols)) {
    case 8: WAVE(8); break;
    case 16: WAVE(16); break;
    case 32: WAVE(32); break;
    case 64: WAVE(64); break;
    case 256: GROUP(256, 1); break;
    case 512: GROUP(512, 1); break;
    default:
      if (a.cols <= 8192) GROUP(1024, 1);
      else GROUP(1024, 2);
  }
#undef WAVE
#undef GROUP
  return hipGetLastError();
}

template <int XT>
hipError_t launch_x(const NormArgs& a, hipStream_t s) {
  if (!a.res) return launch_types<XT, kResNone>(a, s);
  if (a.rt == MOE_DT_BF16) return launch_types<XT, MOE_DT_BF16>(a, s);
  if (a.rt == MOE_DT_F16) return launch_types<XT, MOE_DT_F16>(a, s);
  return launch_types<XT, MOE_DT_F32>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.xt == MOE_DT_BF16) return launch_x<MOE_DT_BF16>(a, s);
  if (a.xt == MOE_DT_F16) return launch_x<MOE_DT_F16>(a, s);
  return launch_x<MOE_DT_F32>(a, s);
}

}  // namespace qmoe

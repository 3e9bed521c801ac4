// Products of a few rows with 4-bit weights (moe_linear): the kernel, built
// for each type of row by k_linear_bf16.hip, k_linear_f16.hip, k_linear_i8.hip.
//
// A workgroup takes NT tiles of 16 weight rows, up to R rows of x and all of k: its
// waves take the tiles' steps of 128 columns in turn, so the workgroup reads one
// contiguous run of memory for each tile, and add their sums up through LDS in wave
// order (no workspace, no atomics).  A lane's 16 bytes of a tile are its operand of four
// 16x16x32 products (lane c = 16*g + r: weight row r, 8 columns of each); the rows of x are
// read in whole stretches and turned into the other operand through the wave's own part of LDS: read as
// operands, a request for each lane, 64 rows of 7168 codes took 58 us for 16.5.
//
// Few rows are bound by the weights' bytes, many by what a compute unit has to do for them, of which none alone is near its
// peak: of 64 rows of bf16 times 7168 x 7168, 16.5 us, by count matrix instructions are 4 us, vector instructions that make operands
// of codes 5 (half of it twice: a wave's operands serve 32 rows), x from the second-level cache 4 and through LDS 4.
// 1 row times 32771 x 7168 25 to 27 us in bf16 (scales of 128, 4.5 to 4.8 TB/s), 26.8 as codes with scales of 32 (4.9), 22.8 with
// scales of 128 (5.3); 16 rows of bf16 times 7168 x 7168 8.0 us; 64 rows times 7168 x 7168 16.5 us in bf16, 11.3 as codes
// (584 TFLOP/s); times 28672 x 7168 59 and 43.
//
// Codes enter the products exactly.  16-bit rows: q goes into the upper
// mantissa bits of 1.0, u = 1 + q/16 (shift, mask, exclusive or: the codes are stored as q ^ 8),
// and sum_j x_j (q_j - z) = 16 (sum_j x_j u_j - (1 + z/16) sum_j x_j), the sums of x
// by one more product, with ones.  8-bit rows: 16 (q - 8) is a signed byte
// already, (q ^ 8) << 4, and sums are whole numbers; those of x are needed only with zero points.
// A group's sum is scaled once, in 32 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmoe_step.h"
#include "k_step.h"
#include "lds_limit.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <int XT>
struct Types {
  typedef u32x4 X;                  // 8 values of x: one chunk of 32 columns, one lane
  typedef f32x4 Acc;
};
template <>
struct Types<MOE_DT_I8> {
  typedef u32x2 X;
  typedef i32x4 Acc;
};

template <int XT>
__device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (XT == MOE_DT_BF16) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  } else {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
}

// One word of codes (q ^ 8 of columns j at bit 4*(j/2) + 16*(j%2)) as 8 numbers 1 + q/16.
template <int XT>
__device__ __forceinline__ u32x4 units(uint32_t w) {
  constexpr int kAt = XT == MOE_DT_BF16 ? 3 : 6;                    // lowest of the four upper mantissa bits
  constexpr uint32_t kMask = 0x000F000Fu << kAt;
  constexpr uint32_t kFlip = (XT == MOE_DT_BF16 ? 0x3F803F80u : 0x3C003C00u) ^ (0x00080008u << kAt);
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int by = kAt - 4 * p;
    r[p] = ((by >= 0 ? w << (by & 31) : w >> (-by & 31)) & kMask) ^ kFlip;
  }
  return r;
}

// The same as 8 signed bytes 16 (q - 8), in the order of columns 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x2 bytes(uint32_t w) { return (u32x2){(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u}; }
// 8 bytes of a row in that order.
__device__ __forceinline__ u32x2 in_order(uint32_t lo, uint32_t hi) {
  return (u32x2){__builtin_amdgcn_perm(hi, lo, 0x05010400u), __builtin_amdgcn_perm(hi, lo, 0x07030602u)};
}

// Reads past the end of a buffer give zeros and cost no traffic: what lies past the last
// column, row or tile is read there.  (Offsets are in the vector operand only, which is what is compared with the end.)
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00027000);
}

// A tile's share of a lane: codes, and (perhaps with its neighbours') its row's scales and zero points.
template <int G, bool Z>
struct Weights {
  u32x4 q;
  u32x2 s;                           // fp16 scales of 128 / G groups
  uint32_t z;                        // bytes z - 8
};

template <int G, bool Z>
__device__ __forceinline__ Weights<G, Z> load_weights(Buffer b, uint32_t tile, uint32_t lane) {
  constexpr int kGroups = 128 / G;
  const uint32_t r = lane & 15;
  Weights<G, Z> w;
  w.q = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, tile + 16 * lane, 0, 0));
  if constexpr (G == 32) w.s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, tile + 1024 + 8 * r, 0, 0));
  else w.s = (u32x2){(uint32_t)__builtin_amdgcn_raw_buffer_load_b32(b, tile + 1024 + (G == 64 ? 4 * r : 4 * (r / 2)), 0, 0), 0};
  w.z = 0;
  if constexpr (Z)
    w.z = __builtin_amdgcn_raw_buffer_load_b32(b, tile + 1024 + 32 * kGroups + (G == 32 ? 4 * r : G == 64 ? 4 * (r / 2) : 4 * (r / 4)), 0, 0);
  return w;
}

// Scale and z - 8 of group i of the lane's row.
template <int G, bool Z>
__device__ __forceinline__ float scale_of(const Weights<G, Z>& w, int i, uint32_t lane) {
  const uint32_t s = G == 128 ? w.s[0] >> (16 * (lane & 1)) : w.s[i / 2] >> (16 * (i % 2));
  return (float)__builtin_bit_cast(_Float16, (uint16_t)s);
}
template <int G, bool Z>
__device__ __forceinline__ int zero_of(const Weights<G, Z>& w, int i, uint32_t lane) {
  const uint32_t z = G == 128 ? w.z >> (8 * (lane & 3)) : G == 64 ? w.z >> (16 * (lane & 1) + 8 * i) : w.z >> (8 * i);
  return (int)(int8_t)z;
}

// How a workgroup is made for up to R rows of x and NT tiles of 16 weight rows.  (12 or 16 waves were not faster for any
// R and NT.)
constexpr int kWaves = 8;
template <int XT, int R, int NT>
struct Shape {
  static constexpr int kXBytes = XT == MOE_DT_I8 ? 1 : 2;
  // A wave takes up to 32 rows.  For more rows waves of the same columns go side by side and read the same weights.
  static constexpr int kRows = R < 32 ? R : 32, kSides = R / kRows, kSteps = kWaves / kSides;
  static constexpr int kMt = (kRows + 15) / 16;                      // 16-row operands of x
  static constexpr int kLanesARow = 8 * kXBytes;                     // 16 bytes of a row's 128 columns a lane
  static constexpr int kRowsALoad = 64 / kLanesARow;
  static constexpr int kLoads = kRows <= kRowsALoad ? 1 : kRows / kRowsALoad;
  static constexpr int kXTile = 1024 * kLoads, kSums = kMt * NT * 1024;
  static constexpr int kLds = kXTile > kSums ? kXTile : kSums;       // of a wave
  // (rows past kRows: whatever lies behind them, in its wave's or a neighbour's part)
  static constexpr int kLdsAll = (kWaves - 1) * kLds + (kLds > 2048 * kXBytes * kMt ? kLds : 2048 * kXBytes * kMt);
  // Tiles in flight, of x and of the weights alike: loads are waited for in the order in which they were issued, so a
  // later x would hold up the weights in front of it.  One row times 4096 x 7168 5.0 us with two, 5.8 with one, 5.3 with
  // three; with more to do for a tile one is enough and its registers are better free: 32 rows of bf16 times 4096 8.4 with
  // two, 7.9 with one.
  static constexpr int kDepth = R < 16 || (R == 16 && (NT == 1 || kXBytes == 1)) ? 2 : 1;
};

// Z: with zero points.  XG: 8-bit rows with a scale for each 128 columns.
template <int XT, int G, int R, int NT, bool Z, bool XG>
__global__ __launch_bounds__(64 * kWaves) void linear_kernel(LinearArgs a) {
  typedef Shape<XT, R, NT> S;
  constexpr int MT = S::kMt, kSteps = S::kSteps, kGroups = 128 / G, kDepth = S::kDepth;
  constexpr bool kInt = XT == MOE_DT_I8;
  constexpr int kXBytes = S::kXBytes;
  constexpr uint32_t kTile = 1024 + 32 * kGroups + (Z ? 16 * kGroups : 0);
  typedef typename Types<XT>::X X;
  extern __shared__ uint8_t lds[];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, r = lane & 15, g = lane >> 4;
  const int kc_n = (a.k + 127) / 128, rt_n = (a.n + 15) / 16;
  const int side = wave / kSteps, step = wave % kSteps;
  const int t0 = blockIdx.y * R + side * S::kRows, rt0 = blockIdx.x * NT;   // (t0 may lie past the last row)
  Buffer tiles[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    tiles[i] = buffer(a.w + (int64_t)(rt0 + i) * kc_n * kTile, rt0 + i < rt_n ? kc_n * kTile : 0);
  // kRows rows of x from t0 on: below 2^31 bytes, as strides are at most 2^24
  constexpr uint32_t kNoRow = 0x80000000u, kNoColumn = 0x7FFFFFF0u;
  const int rows = min(a.rows - t0, S::kRows);
  const Buffer xs = buffer((const uint8_t*)a.x + (rows > 0 ? (int64_t)t0 * a.x_stride * kXBytes : 0),
                           rows > 0 ? (uint32_t)(((rows - 1) * a.x_stride + a.k) * kXBytes) : 0);
  // A load takes whole stretches of rows; the wave's part of LDS turns them into operands.  16 bytes u of row i lie
  // at u ^ i among the row's, so that the 16 rows of an operand are in different banks.
  const uint32_t lrow = lane / S::kLanesARow, unit = lane % S::kLanesARow;
  uint32_t xrow[S::kLoads], trow[MT];                                // trow: the lane's 4 rows of the results
#pragma unroll
  for (int q = 0; q < S::kLoads; ++q) {
    const int i = q * S::kRowsALoad + lrow;
    xrow[q] = i < rows ? i * (uint32_t)a.x_stride * kXBytes : kNoRow;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) trow[m] = (uint32_t)min(t0 + 16 * m + 4 * (int)g, (a.rows - 1) & ~3);
  uint8_t* const mine = lds + wave * S::kLds;
  uint8_t* const put = mine + lrow * (16 * S::kLanesARow);
  const uint8_t* const get = mine + r * (16 * S::kLanesARow);

  Weights<G, Z> w[kDepth][NT];
  u32x4 x[kDepth][S::kLoads];
  f32x4 xg[kDepth][XG ? MT : 1];
  auto load_w = [&](int d, int i) {                                  // of the wave's tile i
    const int kc = step + i * kSteps;
#pragma unroll
    for (int t = 0; t < NT; ++t) w[d][t] = load_weights<G, Z>(tiles[t], kc * kTile, lane);
    if constexpr (XG) {
#pragma unroll
      for (int m = 0; m < MT; ++m) xg[d][m] = *(const f32x4*)(a.xs + min(kc, kc_n - 1) * a.xs_stride + trow[m]);
    }
  };
  auto load_x = [&](int d, int i) {
    const int col = (step + i * kSteps) * 128 + (int)unit * (16 / kXBytes);
    const uint32_t at = col < a.k ? (uint32_t)col * kXBytes : kNoColumn;
#pragma unroll
    for (int q = 0; q < S::kLoads; ++q)
      x[d][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xs, xrow[q] + at, 0, 0));
  };
  // (the lanes of a wave exchange x through its part of LDS, whose operations are done in order)
  auto turn = [&](int d, int i) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const bool half = kInt && (step + i * kSteps) * 128 + (int)unit * 16 + 8 >= a.k;   // (k is a multiple of 8)
#pragma unroll
    for (int q = 0; q < S::kLoads; ++q) {
      u32x4 v = x[d][q];
      if (half) v[2] = 0, v[3] = 0;
      if constexpr (kInt) {                                          // (once for all of the weights' tiles)
        const uint32_t x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];
        const u32x2 a = in_order(x0, x1), b = in_order(x2, x3);
        v = (u32x4){a[0], a[1], b[0], b[1]};
      }
      const uint32_t row = q * S::kRowsALoad + lrow;
      *(u32x4*)(put + q * 1024 + 16 * (unit ^ (row & (S::kLanesARow - 1)))) = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  auto operand = [&](int m, int c) {                                 // 8 columns of row 16 m + r, 32 c + 8 g and on
    if constexpr (kInt) return *(const u32x2*)(get + m * 2048 + 16 * ((2 * c + (g >> 1)) ^ (r & 7)) + 8 * (g & 1));
    else return *(const u32x4*)(get + m * 4096 + 16 * ((4 * c + g) ^ r));
  };
  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = (f32x4){0, 0, 0, 0};

  auto add = [&](int d) {
    [[maybe_unused]] f32x4 part[MT][NT];
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
      if constexpr (!kInt) {
        constexpr uint32_t kOne = XT == MOE_DT_BF16 ? 0x3F803F80u : 0x3C003C00u;
        const u32x4 one = {kOne, kOne, kOne, kOne};
        f32x4 acc[MT][NT], accx[MT];
#pragma unroll
        for (int c = 0; c < G / 32; ++c) {
          const int at = gi * (G / 32) + c;
          u32x4 b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) b[t] = units<XT>(w[d][t].q[at]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const X xv = operand(m, at);
            accx[m] = mma16<XT>(xv, one, c ? accx[m] : (f32x4){0, 0, 0, 0});
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = mma16<XT>(xv, b[t], c ? acc[m][t] : (f32x4){0, 0, 0, 0});
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float s = 16.0f * scale_of(w[d][t], gi, lane);
          const float z = Z ? -1.5f - 0.0625f * (float)zero_of(w[d][t], gi, lane) : -1.5f;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) total[m][t][j] = fmaf(s, fmaf(z, accx[m][j], acc[m][t][j]), total[m][t][j]);
        }
      } else {
        i32x4 acc[MT][NT], accx[MT];
        if constexpr (G == 32) {
          long b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) b[t] = __builtin_bit_cast(long, bytes(w[d][t].q[gi]));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const long xv = __builtin_bit_cast(long, operand(m, gi));
            if constexpr (Z) accx[m] = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, 0x0101010101010101l, (i32x4){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, b[t], (i32x4){0, 0, 0, 0}, 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int c = 0; c < G / 64; ++c) {
            const int at = gi * (G / 32) + 2 * c;
            i32x4 b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const u32x2 b0 = bytes(w[d][t].q[at]), b1 = bytes(w[d][t].q[at + 1]);
              b[t] = (i32x4){(int)b0[0], (int)b0[1], (int)b1[0], (int)b1[1]};
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const u32x2 x0 = operand(m, at), x1 = operand(m, at + 1);
              const i32x4 xv = {(int)x0[0], (int)x0[1], (int)x1[0], (int)x1[1]};
              const i32x4 one = {0x01010101, 0x01010101, 0x01010101, 0x01010101};
              if constexpr (Z) accx[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv, one, c ? accx[m] : (i32x4){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv, b[t], c ? acc[m][t] : (i32x4){0, 0, 0, 0}, 0, 0, 0);
            }
          }
        }
        // Sums and zero points times sums are below 2^23 in size: exact in 32-bit numbers, whose products take a quarter
        // of the time of whole ones'.
        f32x4 sum[MT];
        if constexpr (Z) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[m][j] = (float)accx[m][j];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float s = 0.0625f * scale_of(w[d][t], gi, lane);
          const float z = Z ? -16.0f * (float)zero_of(w[d][t], gi, lane) : 0.0f;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float v = (float)acc[m][t][j];
              if constexpr (Z) v = fmaf(z, sum[m][j], v);
              if constexpr (!XG) total[m][t][j] = fmaf(s, v, total[m][t][j]);
              else part[m][t][j] = gi ? fmaf(s, v, part[m][t][j]) : s * v;
            }
        }
      }
    }
    if constexpr (XG) {                                              // the 128 columns' scale of the rows
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[m][t][j] = fmaf(xg[d][m][j], part[m][t][j], total[m][t][j]);
    }
  };

  const int tiles_n = (kc_n - step + kSteps - 1) / kSteps;            // of this wave (0 where there are fewer than waves)
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    // (in the loop's order: a wait there is for as many loads as may be behind the one it is for on every way to it)
    load_x(d, d);
    __builtin_amdgcn_sched_barrier(0);
    load_w(d, d);
    __builtin_amdgcn_sched_barrier(0);
  }
  int i = 0;
  for (; i + kDepth <= tiles_n; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      // (stages mixed up would need more registers than there are)
      __builtin_amdgcn_sched_barrier(0);
      turn(d, i + d);
      load_x(d, i + d + kDepth);
      __builtin_amdgcn_sched_barrier(0);
      add(d);
      __builtin_amdgcn_sched_barrier(0);
      load_w(d, i + d + kDepth);
    }
  }
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) {
    if (i + d >= tiles_n) break;
    __builtin_amdgcn_sched_barrier(0);
    turn(d, i + d);
    add(d);
  }

  f32x4* const sums = (f32x4*)mine;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[(m * NT + t) * 64 + lane] = total[m][t];
  __syncthreads();
  for (int at = threadIdx.x; at < R * NT * 16; at += 64 * kWaves) {
    // consecutive threads: consecutive weight rows
    const int row = at / (16 * NT) % S::kRows, from = at / (16 * NT) / S::kRows, nn = at % (16 * NT);
    const int m = row / 16, t = nn / 16, l = 16 * (row % 16 / 4) + nn % 16, j = row % 4;
    const int tok = blockIdx.y * R + from * S::kRows + row, n = rt0 * 16 + nn;
    if (tok >= a.rows || n >= a.n) continue;
    const float* part = (const float*)(lds + from * kSteps * S::kLds) + ((m * NT + t) * 64 + l) * 4 + j;
    float v = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) v += part[s * (S::kLds / 4)];
    if (kInt && !XG) v *= a.xs[tok];
    if (a.bias) v += a.bias[n];
    const int64_t to = (int64_t)tok * a.y_stride + n;
    if (a.y_type == MOE_DT_F32) ((float*)a.y)[to] = v;
    else if (a.y_type == MOE_DT_BF16) ((__bf16*)a.y)[to] = (__bf16)v;
    else ((_Float16*)a.y)[to] = (_Float16)v;
  }
}

template <int XT, int G, int R, int NT, bool Z, bool XG>
hipError_t launch_one(const LinearArgs& a, hipStream_t s) {
  typedef Shape<XT, R, NT> S;
  const auto kernel = linear_kernel<XT, G, R, NT, Z, XG>;
  if (S::kLdsAll > 65536) {
    const hipError_t e = raise_dyn_lds((const void*)kernel, 0);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)(((a.n + 15) / 16 + NT - 1) / NT), (unsigned)((a.rows + R - 1) / R));
  kernel<<<grid, dim3(64 * kWaves), S::kLdsAll, s>>>(a);
  return hipGetLastError();
}

template <int XT, int G, int R, int NT>
hipError_t launch_tiles(const LinearArgs& a, hipStream_t s) {
  constexpr bool kInt = XT == MOE_DT_I8;
  if (kInt && a.x_group) return a.zeros ? launch_one<XT, G, R, NT, true, kInt>(a, s) : launch_one<XT, G, R, NT, false, kInt>(a, s);
  return a.zeros ? launch_one<XT, G, R, NT, true, false>(a, s) : launch_one<XT, G, R, NT, false, false>(a, s);
}

// A workgroup of R rows and NT tiles: more of either share what the other's operands cost, in fewer workgroups.
struct Choice {
  int rows, tiles;
  int one, more;                                       // 0.1 us a round for k = 7168: one workgroup a compute unit, and where there are more rounds
};
constexpr Choice kChoices16[] = {{4, 1, 28, 25},   {4, 2, 40, 49},   {4, 4, 83, 98},    {16, 1, 39, 35},   {16, 2, 56, 52},
                                 {16, 4, 86, 100}, {32, 2, 93, 81},  {32, 4, 139, 142}, {64, 4, 250, 250}};
constexpr Choice kChoices8[] = {{8, 1, 24, 24},  {8, 2, 32, 44},  {8, 4, 70, 83},   {16, 1, 26, 26}, {16, 2, 38, 44},
                                {16, 4, 63, 86}, {32, 2, 55, 53}, {32, 4, 93, 100}, {64, 4, 164, 175}};

// The choice whose workgroups, a compute unit at a time, take the least time, as it was measured for k = 7168 without zero
// points or scales of groups of x (other k were not).  Of k = 7168, in one sweep, 64 rows of bf16 times 256
// weight rows: 4.6 us with 4 rows and a tile a workgroup, 12 with 64 and one; times 4096: 10.8 with 16 and 4, 11.5 with 32 and
// 2, 14.9 with 64 and one; times 7168: 16.1 with 32 and 4, 18.6 with 32 and 2, 24.3 with 64 and 4; times 28672: 67.7, 76 (64 and
// 2) and 55.  As codes times 4096: 8.3, 7.7 and 10.0.  One row times 7168: 6.7 with 2 tiles, 6.9 with one, 8.7 with 4.
// Where there are many rounds the last is not full, and the choices are within a tenth of each other.  Groups of 32 have more
// to do for each tile: 48 rows of fp16 times 4096 x 4096 10.1 with 16 and 4, 9.6 with 32 and 2.
template <int XT, int G>
hipError_t launch_group(const LinearArgs& a, int cus, hipStream_t s) {
  constexpr const auto& kChoices = XT == MOE_DT_I8 ? kChoices8 : kChoices16;
  const int64_t tiles = (a.n + 15) / 16;
  int best = 0;
  int64_t least = INT64_MAX;
  for (int i = 0; i < 9; ++i) {
    const Choice& c = kChoices[i];
    const int64_t parts = (a.rows + c.rows - 1) / c.rows, rounds = (parts * ((tiles + c.tiles - 1) / c.tiles) + cus - 1) / cus;
    const int64_t time = rounds * ((rounds == 1 ? c.one : c.more) + (G == 32 ? 4 * c.tiles : 0));
    if (time < least && parts <= 65535) {              // (the grid's second dimension)
      least = time;
      best = i;
    }
  }
  switch (best) {
    case 0: return launch_tiles<XT, G, kChoices[0].rows, 1>(a, s);
    case 1: return launch_tiles<XT, G, kChoices[1].rows, 2>(a, s);
    case 2: return launch_tiles<XT, G, kChoices[2].rows, 4>(a, s);
    case 3: return launch_tiles<XT, G, 16, 1>(a, s);
    case 4: return launch_tiles<XT, G, 16, 2>(a, s);
    case 5: return launch_tiles<XT, G, 16, 4>(a, s);
    case 6: return launch_tiles<XT, G, 32, 2>(a, s);
    case 7: return launch_tiles<XT, G, 32, 4>(a, s);
    default: return launch_tiles<XT, G, 64, 4>(a, s);
  }
}

}  // namespace

template <int XT>
hipError_t launch_linear_type(const LinearArgs& a, int group, int cus, hipStream_t s) {
  if (group == 32) return launch_group<XT, 32>(a, cus, s);
  if (group == 64) return launch_group<XT, 64>(a, cus, s);
  return launch_group<XT, 128>(a, cus, s);
}

}  // namespace qmoe

// The paged 8-bit key/value cache: rotary positions and appending
// (moe_kv_append), reading rows back (moe_kv_read).  Layout and rules in
// include/qmoe_attn.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.hpp"

using namespace qmoe;
using namespace qmoe_dev;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Least power of two s with amax <= 448 s, not below 2^-64.  448 = 1.75 * 2^8,
// so s has amax's exponent minus 8, one more when the mantissa exceeds 1.75.
__device__ __forceinline__ float least_scale(float amax) {
  const uint32_t u = __builtin_bit_cast(uint32_t, amax);
  int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased
  if (e < 127 - 64) e = 127 - 64;
  return __builtin_bit_cast(float, (uint32_t)e << 23);
}

// 1/s of a power of two between 2^-64 and 2^121
__device__ __forceinline__ float inverse_pow2(float s) {
  return __builtin_bit_cast(float, (254u << 23) - __builtin_bit_cast(uint32_t, s));
}

__device__ __forceinline__ bool finite(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u; }

// Sine and cosine of |x| <= pi/4 by their series: the first terms left out are
// below 2^-45 of the sine and 2^-40.
__device__ __forceinline__ void sine_cosine(double x, double* sn, double* cs) {
  const double y = x * x;
  const double s = 1.0 + y * (-1.0 / 6 + y * (1.0 / 120 + y * (-1.0 / 5040 + y * (1.0 / 362880 + y * (-1.0 / 39916800 + y * (1.0 / 6227020800))))));
  const double c = 1.0 + y * (-0.5 + y * (1.0 / 24 + y * (-1.0 / 720 + y * (1.0 / 40320 + y * (-1.0 / 3628800 + y * (1.0 / 479001600))))));
  *sn = x * s;
  *cs = c;
}

// 32 bits of each x that rounded again to fewer (12 of mantissa at most: a
// row's, a code's) give what x itself rounds to.  Those are the nearest 32
// bits, but for those that look like a border between two shorter numbers:
// there x is cut off and the last bit set in place of the bits lost.
template <int N>
__device__ __forceinline__ void to_round_again(const double* x, float* f) {
  uint32_t low = 0xFFFu;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = (float)x[i];
    low = min(low, __builtin_bit_cast(uint32_t, f[i]) & 0xFFFu);
  }
  if (low != 0) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t u = __builtin_bit_cast(uint32_t, f[i]);
    if ((u & 0xFFFu) == 0 && finite(f[i])) {
      if (fabs((double)f[i]) > fabs(x[i])) --u;
      if ((double)f[i] != x[i]) u |= 1;
      f[i] = __builtin_bit_cast(float, u);
    }
  }
}


__device__ __forceinline__ float amax_of(float m, float x) { return finite(x) ? fmaxf(m, fabsf(x)) : m; }

// Code of x (already divided by the scale); not finite -> not a number.
__device__ __forceinline__ uint32_t code2(float a, float b) {
  const float nan = __builtin_nanf("");
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(finite(a) ? a : nan, finite(b) ? b : nan, 0, false) & 0xFFFFu;
}

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  return code2(a, b) | code2(c, d) << 16;
}

// Four codes times r, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  const auto x = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto y = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return code4(x[0] * r, x[1] * r, y[0] * r, y[1] * r);
}

// Maximum over a wave: within 4 lanes, 8, 16, then over its rows of 16.
__device__ __forceinline__ float wave_max(float x) {
  const auto step = [](float v, auto ctrl) {
    const int w = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, true);
    return fmaxf(v, __builtin_bit_cast(float, w));
  };
  x = step(x, std::integral_constant<int, 0xB1>());    // quad_perm 1 0 3 2
  x = step(x, std::integral_constant<int, 0x4E>());    // quad_perm 2 3 0 1
  x = step(x, std::integral_constant<int, 0x141>());   // row_half_mirror
  x = step(x, std::integral_constant<int, 0x140>());   // row_mirror
  return max_rows4(x);
}

template <typename T>
__device__ __forceinline__ void unpack8(const u32x4& v, float* x) {
  x[0] = T::lo(v.x); x[1] = T::hi(v.x); x[2] = T::lo(v.y); x[3] = T::hi(v.y);
  x[4] = T::lo(v.z); x[5] = T::hi(v.z); x[6] = T::lo(v.w); x[7] = T::hi(v.w);
}

template <typename T>
__device__ __forceinline__ u32x4 pack8(const float* x) {
  u32x4 v;
  v.x = T::cvt2(x[0], x[1]); v.y = T::cvt2(x[2], x[3]); v.z = T::cvt2(x[4], x[5]); v.w = T::cvt2(x[6], x[7]);
  return v;
}

__device__ __forceinline__ u32x4 ldg16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// Index in the cache of block `blk` of head hk, on page `page`.
__device__ __forceinline__ int64_t block_in(const KvArgs& a, int page, int blk, int hk) {
  return ((((int64_t)page * a.Hk + hk) << a.lb) + (blk & ((1 << a.lb) - 1)));
}

// One workgroup takes the tokens that one block of one sequence gets, and a
// share (blockIdx.y) of the heads.  Its threads compute the angles of those
// tokens once into LDS, in 64 bits for k, whose codes then fall at the borders
// between them as in 64-bit arithmetic, and rounded to 32 for q; then
// each wave takes one job at a time: a q head (turn), a K head (turn, scale,
// codes) or a V head (scale, codes).  A wave holds 16 tokens of one head in
// registers, so each input is read once and each output written once.  The
// first job's loads are asked for before the angles: with one token it is
// latency that counts.  (With many, asking for each next job's loads while one
// is worked on costs registers and 4% at 2048 tokens of 32 + 8 + 8 heads.)
//
// Bound by memory: 2048 tokens, heads of 128: 50 MB in 13.7 us, 3.7 TB/s (a
// copy of 4 GB reaches 4.7); without a turn 12.5, with all of it in 32 bits 12.9.
// One token 4.9 us, 64 users of up to 3 tokens 6.0: a launch and three loads
// that wait for one another (length, page, scale).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int nb) {
  constexpr int kLanes = D / 16;            // lanes of a row of q or k, 16 columns each
  constexpr int kRows = 64 / kLanes;        // rows a wave takes at once
  constexpr int kSteps = 16 / kRows;
  constexpr int kCh = D / 8;                // V: a lane takes 8 columns of 4 tokens, the words of its columns
  constexpr int kSt = kCh * 4 > 64 ? kCh * 4 / 64 : 1;
  constexpr int kRaw = 2 * kSteps > 4 * kSt ? 2 * kSteps : 4 * kSt;
  __shared__ __attribute__((aligned(16))) float2 turn[16][D / 2 + 1];
  constexpr int kPitch = kLanes + 1;        // (so that neither writes nor reads meet in a bank)
  __shared__ __attribute__((aligned(16))) double2 exact[16][8 * kPitch];   // pair 8 c + j at j * kPitch + c

  const int b = nb == 1 ? blockIdx.x : blockIdx.x / nb, ib = nb == 1 ? 0 : blockIdx.x % nb;
  const Seq s = seq_of(a.kv, b);
  const int pos0 = s.len - s.n;             // may be negative
  const int blk = (pos0 >> 4) + ib;
  const int lo = max(blk * 16, pos0), hi = min(blk * 16 + 16, s.len);
  if (lo >= hi) return;                     // the whole workgroup
  const int f = lo - blk * 16, e = hi - blk * 16;      // slots [f, e) are new
  const int64_t row_of_slot0 = (int64_t)s.row0 + (blk * 16 - pos0);
  const int half = a.rot / 2;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int jobs = a.Hq + 2 * a.kv.Hk;
  const int page = blk < 0 ? -1 : a.kv.table[(int64_t)b * a.kv.table_stride + (blk >> a.kv.lb)];
  const bool held = (unsigned)page < (unsigned)a.kv.n_pages;   // the block is one of the cache's

  // rows of q and k: lane -> (row of the step, 16 columns as two chunks of 8)
  const int c = lane % kLanes, rr = lane / kLanes;
  const bool turned = 16 * c < a.rot;
  const int dA = (!a.inter && turned) ? 8 * c : 16 * c;
  const int dB = (!a.inter && turned) ? half + 8 * c : 16 * c + 8;

  u32x4 raw[kRaw];                          // a job's rows as they come
  float was = 0.f;                          // its block's scale so far
  const auto load = [&](int job) {
    if (job >= jobs) return;
    if (job < a.Hq + a.kv.Hk) {
      const bool is_q = job < a.Hq;
      const uint16_t* src = (const uint16_t*)(is_q ? a.q : a.k) + (int64_t)(is_q ? job : job - a.Hq) * D;
      const int64_t stride = is_q ? a.qs : a.ks;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int n = st * kRows + rr;
        raw[2 * st] = raw[2 * st + 1] = u32x4{0, 0, 0, 0};
        if (n >= f && n < e) {
          const uint16_t* p = src + (row_of_slot0 + n) * stride;
          raw[2 * st] = ldg16(p + dA);
          raw[2 * st + 1] = ldg16(p + dB);
        }
      }
      if (!is_q && held && f > 0) was = a.kv.scales[2 * block_in(a.kv, page, blk, job - a.Hq)];
    } else if (held) {
      const uint16_t* src = (const uint16_t*)a.v + (int64_t)(job - a.Hq - a.kv.Hk) * D;
#pragma unroll
      for (int st = 0; st < kSt; ++st) {
        const int l = st * 64 + lane, ch = l % kCh, g = l / kCh;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = 4 * g + i;
          raw[4 * st + i] = u32x4{0, 0, 0, 0};
          if (g < 4 && n >= f && n < e) raw[4 * st + i] = ldg16(src + (row_of_slot0 + n) * a.vs + 8 * ch);
        }
      }
      if (f > 0) was = a.kv.scales[2 * block_in(a.kv, page, blk, job - a.Hq - a.kv.Hk) + 1];
    }
  };

  int job = blockIdx.y * kWaves + wave;
  load(job);

  if (half > 0) {
    bool has_k = false;                     // whether a K head is among this workgroup's jobs
    for (int j = blockIdx.y * kWaves; j < a.Hq + a.kv.Hk; j += kWaves * gridDim.y) has_k |= j + kWaves > a.Hq;
    // a thread takes one pair of every (256 / 2^sh)th new token
    const int sh = half <= 32 ? 5 : half <= 64 ? 6 : 7, p = threadIdx.x & ((1 << sh) - 1);
    if (p < half) {
      const double w = a.freqs[p] * 0.15915494309189535;       // turns a position
      for (int n = f + (threadIdx.x >> sh); n < e; n += kThreads >> sh) {
        // whole quarter turns off, and sine and cosine of the rest
        const double t = 4.0 * (double)(blk * 16 + n) * w, quarters = rint(t);
        double sn, cs;
        sine_cosine((t - quarters) * 1.5707963267948966, &sn, &cs);
        const int k = (int)(quarters - 4.0 * floor(0.25 * quarters));
        const double s4 = k & 1 ? cs : sn, c4 = k & 1 ? sn : cs;
        const double2 u = make_double2(k == 1 || k == 2 ? -c4 : c4, k >= 2 ? -s4 : s4);
        if (has_k) exact[n][(p & 7) * kPitch + (p >> 3)] = make_double2(u.x * a.rscale, u.y * a.rscale);
        turn[n][p] = make_float2((float)(u.x * a.rscale), (float)(u.y * a.rscale));
      }
    }
    __syncthreads();
  }

  for (bool more = false; job < jobs; job += kWaves * gridDim.y, more = true) {
    if (more) load(job);
    if (job < a.Hq + a.kv.Hk) {
      const bool is_q = job < a.Hq;
      const int h = is_q ? job : job - a.Hq;
      uint16_t* dst = (uint16_t*)(is_q ? a.q_out : a.k_out);
      const int64_t dstride = is_q ? a.qos : a.kos;
      float x[kSteps][16];
      float m = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int n = st * kRows + rr;
        const bool on = n >= f && n < e;
        float* A = x[st];
        float* B = x[st] + 8;
        unpack8<T>(raw[2 * st], A);
        unpack8<T>(raw[2 * st + 1], B);
        if (turned && on && !is_q) {
          const double2* t = &exact[n][c];
#pragma unroll
          for (int j0 = 0; j0 < 8; j0 += 2) {
            // (pair j of the lane's: columns j and 8 + j of its 16, or 2 j and 2 j + 1)
            double v[4];
            float y[4];
#pragma unroll
            for (int j = j0; j < j0 + 2; ++j) {
              const double2 u = t[j * kPitch];
              const double va = a.inter ? x[st][2 * j] : A[j], vb = a.inter ? x[st][2 * j + 1] : B[j];
              v[2 * (j - j0)] = va * u.x - vb * u.y;
              v[2 * (j - j0) + 1] = va * u.y + vb * u.x;
            }
            to_round_again<4>(v, y);
#pragma unroll
            for (int j = j0; j < j0 + 2; ++j) {
              if (a.inter) {
                x[st][2 * j] = y[2 * (j - j0)];
                x[st][2 * j + 1] = y[2 * (j - j0) + 1];
              } else {
                A[j] = y[2 * (j - j0)];
                B[j] = y[2 * (j - j0) + 1];
              }
            }
          }
        } else if (turned && on) {
          const float2* t = &turn[n][8 * c];
          if (a.inter) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 u = t[j], v = t[4 + j];
              const float a0 = A[2 * j], a1 = A[2 * j + 1], b0 = B[2 * j], b1 = B[2 * j + 1];
              A[2 * j] = a0 * u.x - a1 * u.y;
              A[2 * j + 1] = a0 * u.y + a1 * u.x;
              B[2 * j] = b0 * v.x - b1 * v.y;
              B[2 * j + 1] = b0 * v.y + b1 * v.x;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 u = t[j];
              const float a0 = A[j], b0 = B[j];
              A[j] = a0 * u.x - b0 * u.y;
              B[j] = a0 * u.y + b0 * u.x;
            }
          }
        }
        if (on && dst) {
          uint16_t* p = dst + (row_of_slot0 + n) * dstride + (int64_t)h * D;
          *reinterpret_cast<u32x4*>(p + dA) = pack8<T>(A);
          *reinterpret_cast<u32x4*>(p + dB) = pack8<T>(B);
        }
        if (!is_q) {
#pragma unroll
          for (int j = 0; j < 16; ++j) m = amax_of(m, x[st][j]);
        }
      }
      if (is_q || !held) continue;
      const int64_t at = block_in(a.kv, page, blk, h);
      uint8_t* tile = a.kv.codes + at * (32 * D);
      const float now = fmaxf(was, least_scale(wave_max(m)));
      const float inv = inverse_pow2(now);
      if (f > 0 && now > was) {       // earlier tokens of the block: lane c = 16*g + n
        if ((lane & 15) < f) {
          const float r = was * inv;
#pragma unroll
          for (int p = 0; p < D / 64; ++p) {
            u32x4* w = reinterpret_cast<u32x4*>(tile + 1024 * p + 16 * lane);
            u32x4 v = *w;
            v.x = rescale4(v.x, r);
            v.y = rescale4(v.y, r);
            v.z = rescale4(v.z, r);
            v.w = rescale4(v.w, r);
            *w = v;
          }
        }
      }
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int n = st * kRows + rr;
        if (n < f || n >= e) continue;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const float* y = x[st] + 8 * part;
          const int d = part ? dB : dA;
          u32x2 w;
          w.x = code4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
          w.y = code4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
          *reinterpret_cast<u32x2*>(tile + 1024 * (d >> 6) + 16 * (16 * ((d >> 3) & 3) + n) + 8 * ((d >> 5) & 1)) = w;
        }
      }
      if (lane == 0) a.kv.scales[2 * at] = now;
    } else if (held) {
      const int64_t at = block_in(a.kv, page, blk, job - a.Hq - a.kv.Hk);
      uint8_t* tile = a.kv.codes + at * (32 * D) + 16 * D;
      // words that keep bytes of other tokens
      uint32_t old[kSt][8];
#pragma unroll
      for (int st = 0; st < kSt; ++st) {
        const int l = st * 64 + lane, ch = l % kCh, g = l / kCh;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = 8 * ch + j;
          old[st][j] = 0;
          if (g < 4 && (f > 4 * g || e < 4 * g + 4))
            old[st][j] = *reinterpret_cast<const uint32_t*>(tile + 1024 * (d >> 6) + 16 * (16 * g + (d & 15)) + 4 * ((d >> 4) & 3));
        }
      }
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * kSt; ++i) {
        float x[8];
        unpack8<T>(raw[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = amax_of(m, x[j]);
      }
      const float now = fmaxf(was, least_scale(wave_max(m)));
      const float inv = inverse_pow2(now);
      const float r = was * inv;
#pragma unroll
      for (int st = 0; st < kSt; ++st) {
        const int l = st * 64 + lane, ch = l % kCh, g = l / kCh;
        const bool grow = f > 4 * g && now > was;        // holds tokens to be rounded again
        const bool fresh = f < 4 * g + 4 && e > 4 * g;         // gets new tokens
        if (g >= 4 || !(grow || fresh)) continue;
        // bytes of new tokens, and of earlier ones
        const int nf = min(max(f - 4 * g, 0), 4), ne = min(max(e - 4 * g, 0), 4);
        const uint32_t below = nf >= 4 ? 0xFFFFFFFFu : (1u << (8 * nf)) - 1u;
        const uint32_t upto = ne >= 4 ? 0xFFFFFFFFu : (1u << (8 * ne)) - 1u;
        const uint32_t is_new = upto & ~below;
        float x[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack8<T>(raw[4 * st + i], x[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = 8 * ch + j;
          uint32_t word = code4(x[0][j] * inv, x[1][j] * inv, x[2][j] * inv, x[3][j] * inv);
          word = (word & is_new) | (old[st][j] & ~is_new);
          if (grow) word = (word & ~below) | (rescale4(old[st][j], r) & below);
          *reinterpret_cast<uint32_t*>(tile + 1024 * (d >> 6) + 16 * (16 * g + (d & 15)) + 4 * ((d >> 4) & 3)) = word;
        }
      }
      if (lane == 0) a.kv.scales[2 * at + 1] = now;
    }
  }
}

// Whether codes times this scale (the wave's) may leave the row type's range, and then two
// values of which an infinite one becomes the type's largest (a code is never
// infinite: its row was finite, at most half a step of the code away).
template <typename T>
__device__ __forceinline__ bool may_leave(float scale) {
  return (__builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, scale)) >> 23 & 0xFF) >= 127 + T::kOver;
}

template <typename T>
__device__ __forceinline__ uint32_t kept_finite(uint32_t w) {
  const uint32_t lo = (w & 0x7FFFu) == T::kExpOne ? 1u : 0u, hi = (w >> 16 & 0x7FFFu) == T::kExpOne ? 0x10000u : 0u;
  return w - lo - hi;
}

// One wave takes one block of one sequence and head: the K codes go out as
// they lie (a lane holds 8 consecutive columns of one token), the V codes
// through a transposing tile in LDS, so that rows are written 16 bytes a lane.
// Bound by memory: 7 contexts of up to 8191, 8 heads of 64: 75 MB in 13.5 us,
// 5.6 TB/s; 2048 positions, 8 heads of 128 (12.6 MB) in 4.9 us.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a, int nb) {
  constexpr int kPad = 8;
  __shared__ __attribute__((aligned(16))) uint16_t vt[kWaves][16][D + kPad];
  const int b = nb == 1 ? blockIdx.x : blockIdx.x / nb, ib = nb == 1 ? 0 : blockIdx.x % nb;
  const Seq s = seq_of(a.kv, b);
  const int pos0 = s.len - s.n;
  const int blk = (pos0 >> 4) + ib;
  const int lo = max(blk * 16, pos0), hi = min(blk * 16 + 16, s.len);
  if (lo >= hi) return;
  const int f = lo - blk * 16, e = hi - blk * 16;
  const int64_t row_of_slot0 = (int64_t)s.row0 + (blk * 16 - pos0);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n = lane & 15, g = lane >> 4;
  const int h = blockIdx.y * kWaves + wave;
  if (h >= a.kv.Hk) return;
  const int64_t at = blk < 0 ? -1 : block_of(a.kv, b, blk, h);
  const uint8_t* tile = a.kv.codes + (at < 0 ? 0 : at) * (32 * D);
  float sk = 1.f, sv = 1.f;
  if (at >= 0) {
    sk = a.kv.scales[2 * at];
    sv = a.kv.scales[2 * at + 1];
  }
  u32x4 kw[D / 64], vw[D / 64];
#pragma unroll
  for (int p = 0; p < D / 64; ++p) {
    kw[p] = vw[p] = u32x4{0, 0, 0, 0};
    if (at >= 0) {
      kw[p] = *reinterpret_cast<const u32x4*>(tile + 1024 * p + 16 * lane);
      vw[p] = *reinterpret_cast<const u32x4*>(tile + 16 * D + 1024 * p + 16 * lane);
    }
  }
  const bool on = n >= f && n < e;
  if (on) {
    uint16_t* p = (uint16_t*)a.k_out + (row_of_slot0 + n) * a.kos + (int64_t)h * D + 8 * g;
    const bool k_over = may_leave<T>(sk);
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      u32x4 x = dec8<T>(kw[q].x, kw[q].y, sk), y = dec8<T>(kw[q].z, kw[q].w, sk);
      if (k_over) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = kept_finite<T>(x[i]);
          y[i] = kept_finite<T>(y[i]);
        }
      }
      *reinterpret_cast<u32x4*>(p + 64 * q) = x;
      *reinterpret_cast<u32x4*>(p + 64 * q + 32) = y;
    }
  }
  const bool v_over = may_leave<T>(sv);
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t word = w == 0 ? vw[q].x : w == 1 ? vw[q].y : w == 2 ? vw[q].z : vw[q].w;
      uint32_t x = T::dec2(word, sv, false), y = T::dec2(word, sv, true);
      if (v_over) {
        x = kept_finite<T>(x);
        y = kept_finite<T>(y);
      }
      const int d = 64 * q + 16 * w + n;
      vt[wave][4 * g][d] = (uint16_t)x;
      vt[wave][4 * g + 1][d] = (uint16_t)(x >> 16);
      vt[wave][4 * g + 2][d] = (uint16_t)y;
      vt[wave][4 * g + 3][d] = (uint16_t)(y >> 16);
    }
  }
  __builtin_amdgcn_wave_barrier();          // the tile is the wave's own
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  constexpr int kCh = D / 8;
#pragma unroll
  for (int i = lane; i < 16 * kCh; i += 64) {
    const int m = i / kCh, ch = i % kCh;
    if (m < f || m >= e) continue;
    *reinterpret_cast<u32x4*>((uint16_t*)a.v_out + (row_of_slot0 + m) * a.vos + (int64_t)h * D + 8 * ch) =
        *reinterpret_cast<const u32x4*>(&vt[wave][m][8 * ch]);
  }
}

// Blocks of 16 positions that n consecutive ones can touch.
int blocks_of(int n) { return (n + 30) / 16; }

}  // namespace

namespace qmoe {

hipError_t launch_kv_append(const AppendArgs& a, int dtype, int cus, hipStream_t s) {
  const int nb = blocks_of(a.kv.cu ? a.kv.max_new : a.kv.per_seq);
  const int64_t items = (int64_t)a.kv.B * nb;
  const int jobs = a.Hq + 2 * a.kv.Hk;
  // few tokens: a wave per job, so that the heads' latencies overlap; many:
  // a workgroup takes all heads and its angles serve them all.  4 workgroups a
  // compute unit: 2048 tokens 18.0 us a call (1: 22.2, 2: 19.0, 3: 18.5, 8: 20.2)
  int64_t gy = (4ll * cus + items - 1) / items;
  const int most = (jobs + kWaves - 1) / kWaves;
  if (gy > most) gy = most;
  void (*fn)(AppendArgs, int) = nullptr;
  const bool bf = dtype == 0;
  switch (a.kv.D) {
    case 64: fn = bf ? append_kernel<Bf16, 64> : append_kernel<F16, 64>; break;
    case 128: fn = bf ? append_kernel<Bf16, 128> : append_kernel<F16, 128>; break;
    default: fn = bf ? append_kernel<Bf16, 256> : append_kernel<F16, 256>; break;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)items, (unsigned)gy), dim3(kThreads), 0, s, a, nb);
  return hipGetLastError();
}

hipError_t launch_kv_read(const ReadArgs& a, int dtype, hipStream_t s) {
  const int nb = blocks_of(a.kv.cu ? a.kv.max_new : a.kv.per_seq);
  void (*fn)(ReadArgs, int) = nullptr;
  const bool bf = dtype == 0;
  switch (a.kv.D) {
    case 64: fn = bf ? read_kernel<Bf16, 64> : read_kernel<F16, 64>; break;
    case 128: fn = bf ? read_kernel<Bf16, 128> : read_kernel<F16, 128>; break;
    default: fn = bf ? read_kernel<Bf16, 256> : read_kernel<F16, 256>; break;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.kv.B * (int64_t)nb), (unsigned)((a.kv.Hk + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, s, a, nb);
  return hipGetLastError();
}

}  // namespace qmoe

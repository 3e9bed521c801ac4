// Host side of the 4-bit products (include/qmoe_step.h): the quantizer and the packer of
// their weights.  fp64 arithmetic, built without contraction into fused multiply-adds.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <string>
#include <thread>
#include <vector>

#include "../../include/qmoe_step.h"
#include "half.h"
#include "qmoe_internal.h"

using namespace qmoe;

namespace {

bool shape_ok(int64_t n, int64_t k, int32_t group) {
  return n >= 1 && n <= (1 << 24) && k >= 8 && k <= (1 << 20) && k % 8 == 0 && (group == 32 || group == 64 || group == 128);
}

int bad(const char* who, const std::string& what) { return fail(MOE_ERR_INVALID_ARG, std::string(who) + ": " + what); }

// f(first, last) over [0, n) cut among threads.
template <typename F>
void in_threads(int64_t n, int n_threads, int64_t least, F f) {
  int64_t t = n_threads > 0 ? n_threads : (int64_t)std::thread::hardware_concurrency();
  t = std::max<int64_t>(1, std::min(t, n / std::max<int64_t>(least, 1)));
  std::vector<std::thread> threads;
  int64_t at = 0;
  try {
    threads.reserve((size_t)t);
    for (int64_t i = 1; i < t; ++i) {
      const int64_t to = n * i / t;
      threads.emplace_back(f, at, to);
      at = to;
    }
  } catch (...) {
    // (no more threads to be had: the rest is done here)
  }
  f(at, n);
  for (auto& th : threads) th.join();
}

constexpr int64_t kLeast = 1 << 18;    // values worth a thread

int quantize(const float* w, int64_t n, int64_t k, int32_t group, uint8_t* codes, uint16_t* scales, uint8_t* zeros, int n_threads) {
  static const char* who = "moe_linear_quantize";
  const int64_t gn = (k + group - 1) / group;
  // first only looked through: nothing is written unless all of it can be
  for (int pass = 0; pass < 2; ++pass) {
    std::atomic<int> wrong{0};
    in_threads(n, n_threads, kLeast / k + 1, [&](int64_t r0, int64_t r1) {
      for (int64_t r = r0; r < r1; ++r)
        for (int64_t g = 0; g < gn; ++g) {
          const float* x = w + r * k + g * group;
          const int64_t m = std::min<int64_t>(group, k - g * group);
          double lo = 0, hi = 0;
          for (int64_t j = 0; j < m; ++j) {
            if (!isfinite(x[j])) wrong |= 1;
            lo = std::min(lo, (double)x[j]);
            hi = std::max(hi, (double)x[j]);
          }
          const uint16_t h = f64_to_f16_rne(zeros ? (hi - lo) / 15.0 : (std::max(-lo, hi) + 0.0) / 7.0);    // (+0 for zeros)
          const double s = f16_value(h);
          if (!isfinite(s)) wrong |= 2;
          if (pass == 0) continue;
          int z = 8;
          if (zeros && s > 0) z = (int)std::min(15.0, std::max(0.0, floor(-lo / s + 0.5)));
          for (int64_t j = 0; j < m; ++j)
            codes[r * k + g * group + j] = s > 0 ? (uint8_t)std::min(15.0, std::max(0.0, floor(x[j] / s + 0.5) + z)) : 8;
          scales[r * gn + g] = h;
          if (zeros) zeros[r * gn + g] = (uint8_t)z;
        }
    });
    if (wrong & 1) return bad(who, "non-finite weight");
    if (wrong & 2) return bad(who, "an fp16 scale is out of range");
  }
  return MOE_OK;
}

int pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t n, int64_t k, int32_t group, uint8_t* out,
         int n_threads) {
  static const char* who = "moe_linear_pack";
  const int64_t gn = (k + group - 1) / group, kc_n = (k + 127) / 128, rt_n = (n + 15) / 16;
  const int gt = 128 / group;
  std::atomic<int> wrong{0};
  in_threads(n, n_threads, kLeast / k + 1, [&](int64_t r0, int64_t r1) {
    uint8_t any = 0;
    for (int64_t i = r0 * k; i < r1 * k; ++i) any |= codes[i];
    for (int64_t i = r0 * gn; i < r1 * gn; ++i) {
      if ((scales[i] & 0x7C00) == 0x7C00) wrong |= 2;
      if (zeros) any |= zeros[i];
    }
    if (any > 15) wrong |= 1;
  });
  if (wrong & 1) return bad(who, "codes and zero points must be at most 15");
  if (wrong & 2) return bad(who, "non-finite scale");
  const int64_t tile = 1024 + 32 * gt + (zeros ? 16 * gt : 0);
  in_threads(rt_n, n_threads, kLeast / (16 * k) + 1, [&](int64_t t0, int64_t t1) {
    for (int64_t rt = t0; rt < t1; ++rt)
      for (int64_t kc = 0; kc < kc_n; ++kc) {
        uint8_t* o = out + (rt * kc_n + kc) * tile;
        memset(o, 0, tile);                        // codes of 8, scales of 0, zero points of 8
        for (int r = 0; r < 16 && rt * 16 + r < n; ++r) {
          const int64_t row = rt * 16 + r;
          const uint8_t* q = codes + row * k;
          for (int b = 0; b < 16; ++b) {           // 8 columns: word b / 4 of lane 16 * (b % 4) + r
            const int64_t col = kc * 128 + 8 * b;
            if (col >= k) break;
            uint32_t v = 0;
            for (int j = 0; j < 8; ++j) v |= (uint32_t)(q[col + j] ^ 8) << (4 * (j / 2) + 16 * (j % 2));
            memcpy(o + 16 * (16 * (b % 4) + r) + 4 * (b / 4), &v, 4);
          }
          for (int i = 0; i < gt && kc * gt + i < gn; ++i) {
            memcpy(o + 1024 + 2 * gt * r + 2 * i, scales + row * gn + kc * gt + i, 2);
            if (zeros) o[1024 + 32 * gt + gt * r + i] = (uint8_t)(zeros[row * gn + kc * gt + i] - 8);
          }
        }
      }
  });
  return MOE_OK;
}

}  // namespace

extern "C" int moe_linear_quantize(const float* w, int64_t n, int64_t k, int32_t group, uint8_t* codes, uint16_t* scales,
                                   uint8_t* zeros, int n_threads) {
  clear_error();
  static const char* who = "moe_linear_quantize";
  if (!shape_ok(n, k, group)) return bad(who, "n must be in [1, 2^24], k a multiple of 8 in [8, 2^20], group 32, 64 or 128");
  if (!w || !codes || !scales) return bad(who, "w, codes or scales is NULL");
  return quantize(w, n, k, group, codes, scales, zeros, n_threads);
}

extern "C" size_t moe_linear_packed_bytes(int64_t n, int64_t k, int32_t group, int with_zeros) {
  if (!shape_ok(n, k, group)) return 0;
  return (size_t)((n + 15) / 16) * ((k + 127) / 128) * (1024 + (128 / group) * (with_zeros ? 48 : 32));
}

extern "C" int moe_linear_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t n, int64_t k,
                               int32_t group, void* out, size_t out_bytes, int n_threads) {
  clear_error();
  static const char* who = "moe_linear_pack";
  if (!shape_ok(n, k, group)) return bad(who, "n must be in [1, 2^24], k a multiple of 8 in [8, 2^20], group 32, 64 or 128");
  if (!codes || !scales || !out) return bad(who, "codes, scales or out is NULL");
  if (out_bytes < moe_linear_packed_bytes(n, k, group, zeros != nullptr)) return bad(who, "out_bytes too small");
  return pack(codes, scales, zeros, n, k, group, (uint8_t*)out, n_threads);
}

// Launch interface of the step kernels (k_norm.hip, k_linear*.hip, k_pages.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmoe {

// moe_norm (include/qmoe_step.h); types are MOE_DT_*, null pointers: absent.
struct NormArgs {
  const void *x, *res, *w;
  void *sum, *out;
  int8_t* codes;
  float* scales;
  int64_t xs, rs, ss, os, cs, scs;
  int rows, heads, cols, group;     // group 0: the whole vector
  int xt, rt, wt, ot;
  float eps;
  double per_col;                   // 1 / cols
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
// Threads that take a vector: lanes of a wave for up to 512 columns, else a workgroup.
inline int norm_threads(int cols) {
  return cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 512 ? 64 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
}

// moe_linear.
struct LinearArgs {
  const uint8_t* w;
  const float* bias;
  const void* x;
  const float* xs;
  void* y;
  int64_t x_stride, xs_stride, y_stride;
  int n, k, rows, y_type;
  int zeros;
  int x_group;                      // 0: one scale a row
};
hipError_t launch_linear(const LinearArgs& a, int x_type, int group, int cus, hipStream_t s);

// A pool and the rows of a page table.
struct PagesArgs {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int64_t stride;
  int n_pages, seqs, per_seq, shift;   // page_tokens = 1 << shift
};
hipError_t launch_resize(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, hipStream_t s);

// Caches of one launch that copies pages, by value.
constexpr int kCachesALaunch = 64;
struct PageCopy {
  uint8_t* codes[kCachesALaunch];
  float* scales[kCachesALaunch];
  int32_t heads[kCachesALaunch];
  int32_t block[kCachesALaunch];       // bytes of one block of 16 positions of one head
};
// What the first launch of a fork leaves for the second, a list of: the row, its
// parent (-1: not forked after all), the page to copy from (-1: none) and to (-1: none), and the
// number of blocks to copy.  Its length lies in front of it.
struct ForkJob {
  int32_t row, parent, src, dst, blocks;
};
constexpr size_t kForkHead = 16;
hipError_t launch_fork(const PagesArgs& a, const int32_t* from, int32_t* missing, void* ws, const PageCopy* c,
                       int n_caches, int cus, hipStream_t s);
// ws: int32: pages that move, pages held, 2 unused; [n_pages] number among the moving pages of those from the held
// ones' number on (-1: none); [n_pages] where they go to; [n_pages] where they come from.
hipError_t launch_compact(const PagesArgs& a, int32_t* held, int32_t* ws, const PageCopy* c, int n_caches, int cus,
                          hipStream_t s);

}  // namespace qmoe

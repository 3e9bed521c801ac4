// Pages of a key/value cache kept on the GPU (moe_kv_resize, moe_kv_fork,
// moe_kv_compact).
//
// What has to be decided is small (lengths, one count of holders a page) and
// goes one after the other (rows take free pages in order), so one workgroup
// decides it: sums over rows in LDS, free pages by counting through refs, 16
// stretches of it at once.  There is no list of free pages: the lowest free ids are taken, whatever
// order they were given back in, so that results do not depend on the order of
// atomics.  Page contents are copied by a second launch over the whole card.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "k_step.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct Scratch {
  int32_t wave[2][kWaves];
};

// Sums of v over the threads before this one and over all of them.  `which` alternates between calls, so that one barrier
// a call is enough.
__device__ __forceinline__ int scan(Scratch& s, int which, int v, int* all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 63) s.wave[which][wave] = sum;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int o = s.wave[which][i];
    before += i < wave ? o : 0;
    total += o;
  }
  *all = total;
  return before + sum - v;
}

// Which ids of a window of 4096 * S are free: bit 4 i + c of a lane is that of id first_id(base, i) + c.
template <int S>
struct Free {
  static constexpr int kWindow = kThreads * 4 * S;
  uint32_t bits;
};

template <int S>
__device__ __forceinline__ uint32_t first_id(int base, int i) {
  return base + (((int)threadIdx.x / 64 * S + i) * 64 + (int)threadIdx.x % 64) * 4;
}

// (ids past the pool are not free)
template <int S>
__device__ __forceinline__ Free<S> load_free(const PagesArgs& a, int base) {
  i32x4 v[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const uint32_t id = first_id<S>(base, i);
    v[i] = (i32x4){-1, -1, -1, -1};
    if (id + 4 <= (uint32_t)a.n_pages) {
      v[i] = *(const i32x4*)(a.refs + id);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (id + c < (uint32_t)a.n_pages) v[i][c] = a.refs[id + c];
    }
  }
  Free<S> r{0};
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) r.bits |= (uint32_t)(v[i][c] == 0) << (4 * i + c);
  return r;
}

// How many ids of the wave's part `want` says yes to.
template <int S, typename Want>
__device__ __forceinline__ int count(int base, const Free<S>& r, Want want) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const uint32_t id = first_id<S>(base, i);
#pragma unroll
    for (int c = 0; c < 4; ++c) n += __popcll(__ballot(want(id + c, (r.bits >> (4 * i + c)) & 1)));
    __builtin_amdgcn_sched_barrier(0);         // (one step's ballots at a time: they are scalar registers)
  }
  return n;
}

// f(id, yes, rank) for every id of the wave's part; rank is `first` and the number of yeses before it.
template <int S, typename Want, typename F>
__device__ __forceinline__ void each(int base, const Free<S>& r, int first, Want want, F f) {
  const int lane = threadIdx.x % 64;
  const uint64_t below = (1ull << lane) - 1;
  uint32_t bits = r.bits;
  asm volatile("" : "+v"(bits));               // (or all ballots are kept from one call to the next, in too many registers)
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const uint32_t id = first_id<S>(base, i);
    uint64_t yes[4];
    int rank = first;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      yes[c] = __ballot(want(id + c, (bits >> (4 * i + c)) & 1));
      rank += __popcll(yes[c] & below);
      first += __popcll(yes[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool is = (yes[c] >> lane) & 1;
      f(id + c, is, rank);
      rank += is;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A wave's number in every lane to the sum of those before it.
__device__ __forceinline__ int scan_waves(Scratch& s, int which, int v, int* all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  if (lane == 0) s.wave[which][wave] = v;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int o = s.wave[which][i];
    before += i < wave ? o : 0;
    total += o;
  }
  *all = total;
  return before;
}

constexpr int kList = 4096;        // free pages listed at a time

// Numbers of LDS: sums of the rows' needs and two more numbers a row, and a list of free pages.
struct Rows {
  int32_t *needs, *x, *y, *list;
  __device__ Rows(int32_t* lds, int seqs) : needs(lds + kList), x(needs + seqs), y(x + seqs), list(lds) {}
};
inline size_t rows_lds(int seqs) { return ((size_t)kList + 3 * (size_t)seqs) * 4; }

// Gives the rows whose summed needs fit the lowest free pages, in order: give(first, n) is called with pages of ranks
// first .. first + n - 1 in the list.  Returns how many pages the rows were given.  r: the free pages of the first window.
template <int S, typename Give>
__device__ __forceinline__ int grant(const PagesArgs& a, Scratch& s, const Rows& rows, int total, Free<S>& r, Give give) {
  constexpr int kWindow = Free<S>::kWindow;
  if (total == 0) return 0;
  const auto is_free = [](uint32_t, bool yes) { return yes; };
  __shared__ int32_t fits;
  int free_pages = 0, mine = 0, before = 0, which = 0;
  for (int base = 0; base < a.n_pages && free_pages < total; base += kWindow) {
    if (base) r = load_free<S>(a, base);
    mine = count(base, r, is_free);
    int all;
    before = scan_waves(s, which, mine, &all);
    which ^= 1;
    free_pages += all;
  }
  int granted = total;
  if (free_pages < total) {
    if (threadIdx.x == 0) fits = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < a.seqs; b += kThreads)      // (the last of the sums that fit)
      if (rows.needs[b] <= free_pages && (b + 1 == a.seqs || rows.needs[b + 1] > free_pages)) fits = rows.needs[b];
    __syncthreads();
    granted = fits;
  }
  const bool one = a.n_pages <= kWindow;
  int passed = 0;                                             // free pages of the windows before
  for (int base = 0; passed < granted; base += kWindow) {
    int all = free_pages;
    if (!one) {
      r = load_free<S>(a, base);
      mine = count(base, r, is_free);
      before = scan_waves(s, which, mine, &all);
      which ^= 1;
    }
    const int last = min(granted, passed + all);
    for (int first = passed; first < last; first += kList) {
      const int n = min(kList, last - first);
      if (passed + before < first + n && passed + before + mine > first)
        each(base, r, passed + before, is_free, [&](uint32_t id, bool yes, int rank) {
          if (yes && rank >= first && rank < first + n) {
            rows.list[rank - first] = id;
            a.refs[id] = 1;
          }
        });
      __syncthreads();
      give(first, n);
      if (first + n < granted) __syncthreads();               // (the list is written again)
    }
    passed += all;
  }
  return granted;
}

__device__ __forceinline__ int length(const PagesArgs& a, int v) { return min(max(v, 0), a.per_seq << a.shift); }
__device__ __forceinline__ int pages(const PagesArgs& a, int len) { return (len + (1 << a.shift) - 1) >> a.shift; }
__device__ __forceinline__ bool in_pool(const PagesArgs& a, int p) { return p >= 0 && p < a.n_pages; }

// Entries from..to-1 of a row given back, by `lanes` threads of which this is number `lane`.
__device__ __forceinline__ void release(const PagesArgs& a, int b, int from, int to, int lane, int lanes) {
  int32_t* row = a.table + b * a.stride;
  for (int j = from + lane; j < to; j += lanes) {
    const int p = row[j];
    row[j] = -1;
    if (in_pool(a, p)) atomicSub(a.refs + p, 1);
  }
}

// The rows' pages given back by the whole card, where there may be many: thousands of scattered counts take one
// compute unit 10 us and more.
__global__ __launch_bounds__(256) void release_kernel(PagesArgs a, const int32_t* new_lens) {
  const int b = blockIdx.y, old = a.lens[b], to = new_lens[b];
  if (to < 0) return;
  release(a, b, pages(a, length(a, to)), pages(a, length(a, old)), blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

template <int S>
__global__ __launch_bounds__(kThreads) void resize_kernel(PagesArgs a, const int32_t* new_lens, int32_t* missing, bool released) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  const Rows rows(lds, a.seqs);                                // x: pages held, y: pages wanted
  Free<S> r = load_free<S>(a, 0);                                         // (for the case that none is given back)
  int need_all = 0, which = 0;
  bool drops = false;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int have = 0, want = 0;
    if (b < a.seqs) {
      const int old = a.lens[b], to = new_lens[b];
      have = pages(a, length(a, old));
      want = to < 0 ? have : pages(a, length(a, to));
      rows.x[b] = have;
      rows.y[b] = want;
    }
    drops |= want < have;
    int all;
    const int before = scan(s, which, max(want - have, 0), &all);
    which ^= 1;
    if (b < a.seqs) rows.needs[b] = need_all + before + max(want - have, 0);
    need_all += all;
  }
  // 16 threads a row, or as many as there are for fewer than 64 rows
  int lanes = 16;
  while (lanes < kThreads && lanes * a.seqs < kThreads) lanes *= 2;
  const int group = threadIdx.x / lanes, groups = kThreads / lanes, lane = threadIdx.x % lanes;
  if (__syncthreads_or(drops && !released)) {
    for (int b = group; b < a.seqs; b += groups) release(a, b, rows.y[b], rows.x[b], lane, lanes);
    __threadfence();
    __syncthreads();
    r = load_free<S>(a, 0);
  }
  const int granted = grant(a, s, rows, need_all, r, [&](int first, int n) {
    for (int b = group; b < a.seqs; b += groups) {
      const int end = rows.needs[b], begin = b ? rows.needs[b - 1] : 0;
      if (end <= first || begin >= first + n) continue;
      int32_t* to = a.table + b * a.stride + rows.x[b] - begin;
      for (int i = max(begin, first) + lane; i < min(end, first + n); i += lanes) to[i] = rows.list[i - first];
    }
  });
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    const int to = new_lens[b], end = rows.needs[b], need = end - (b ? rows.needs[b - 1] : 0);
    if (to >= 0 && (need == 0 || end <= granted)) a.lens[b] = length(a, to);
  }
  if (missing && threadIdx.x == 0) *missing = need_all - granted;
}

template <int S>
__global__ __launch_bounds__(kThreads) void fork_kernel(PagesArgs a, const int32_t* from, int32_t* missing, int32_t* head,
                                                        ForkJob* jobs) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  const Rows rows(lds, a.seqs);                                // x: the row's job (-1: none), y: its new length (-1: as it is)
  Free<S> r = load_free<S>(a, 0);
  int sums = 0, which = 0;                                     // jobs, and in the upper half needs, of the rows before
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0, len = 0;
    ForkJob job{b, -1, -1, -1, 0};
    if (b < a.seqs) {
      const int p = from[b], own = length(a, a.lens[b]);
      if (p >= 0 && p < a.seqs) {
        len = length(a, a.lens[p]);
        const int rest = len & ((1 << a.shift) - 1);
        if (len > 0 && (p == b ? rest > 0 : own == 0)) {
          if (rest) {
            const int last = a.table[p * a.stride + (len >> a.shift)];
            job.src = in_pool(a, last) ? last : -1;
            // (a page of its own already needs no other)
            need = p != b || (job.src >= 0 && a.refs[job.src] > 1);
            job.blocks = (rest + 15) / 16;
          }
          if (p != b || need) job.parent = p;
        }
      }
    }
    int all;
    const int before = sums + scan(s, which, (job.parent >= 0) | need << 16, &all);
    which ^= 1;
    sums += all;
    if (job.parent >= 0) jobs[before & 0xFFFF] = job;
    if (b < a.seqs) {
      rows.needs[b] = (before >> 16) + need;
      rows.x[b] = job.parent >= 0 ? before & 0xFFFF : -1;
      rows.y[b] = job.parent >= 0 && job.parent != b ? len : -1;
    }
  }
  const int need_all = sums >> 16;
  __threadfence();
  __syncthreads();
  const int granted = grant(a, s, rows, need_all, r, [&](int first, int n) {
    for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
      const int end = rows.needs[b], begin = b ? rows.needs[b - 1] : 0;
      if (end > begin && begin >= first && begin < first + n) jobs[rows.x[b]].dst = rows.list[begin - first];
    }
  });
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    if (rows.x[b] < 0) continue;
    const int end = rows.needs[b], need = end - (b ? rows.needs[b - 1] : 0);
    if (need && end > granted) jobs[rows.x[b]].parent = -1;
    else if (rows.y[b] >= 0) a.lens[b] = rows.y[b];
  }
  if (threadIdx.x == 0) {
    *head = sums & 0xFFFF;
    if (missing) *missing = need_all - granted;
  }
}

constexpr int kCopyThreads = 256, kCopyUnroll = 8;

// n runs of 16-byte units, `run` long, `pitch` apart, by the workgroups part of parts.
__device__ __forceinline__ void copy_runs(uint8_t* dst, const uint8_t* src, int n, int run, int pitch, int part, int parts) {
  const int total = n * run;
  for (int i0 = part * kCopyThreads * kCopyUnroll; i0 < total; i0 += parts * kCopyThreads * kCopyUnroll) {
    u32x4 v[kCopyUnroll];
    int64_t at[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int i = min(i0 + u * kCopyThreads + (int)threadIdx.x, total - 1);
      at[u] = n == 1 ? (int64_t)i * 16 : ((int64_t)(i / run) * pitch + i % run) * 16;
      v[u] = *(const u32x4*)(src + at[u]);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads + (int)threadIdx.x < total) *(u32x4*)(dst + at[u]) = v[u];
  }
}

// Blocks 0 .. blocks-1 of every head of page src to page dst of cache c.
__device__ __forceinline__ void copy_page(const PagesArgs& a, const PageCopy& c, int cache, int src, int dst, int blocks, int part,
                                          int parts) {
  const int per = 1 << (a.shift - 4), heads = c.heads[cache], block = c.block[cache];
  const int64_t page = (int64_t)heads * per * block;
  uint8_t* codes = c.codes[cache];
  if (blocks == per) copy_runs(codes + dst * page, codes + src * page, 1, heads * per * (block / 16), 0, part, parts);
  else copy_runs(codes + dst * page, codes + src * page, heads, blocks * (block / 16), per * (block / 16), part, parts);
  if (part == 0) {
    float* scales = c.scales[cache];
    for (int i = threadIdx.x; i < heads * blocks * 2; i += kCopyThreads) {
      const int at = i / (blocks * 2) * (per * 2) + i % (blocks * 2);
      scales[(int64_t)dst * heads * per * 2 + at] = scales[(int64_t)src * heads * per * 2 + at];
    }
  }
}

// Workgroups that share a page of a cache, where there are more of them than pages.
__device__ __forceinline__ int parts_of(int units) { return max(1, (int)gridDim.x / max(units, 1)); }

__global__ __launch_bounds__(kCopyThreads) void fork_copy_kernel(PagesArgs a, const int32_t* head, const ForkJob* jobs, PageCopy c,
                                                                 int n_caches, bool first) {
  const int units = *head * n_caches, parts = parts_of(units);
  for (int w = blockIdx.x; w < units * parts; w += gridDim.x) {
    const int unit = w / parts, part = w % parts;
    const ForkJob job = jobs[unit / n_caches];
    const int cache = unit % n_caches;
    if (job.parent < 0) continue;
    if (job.src >= 0 && job.dst >= 0 && c.heads[cache] > 0) copy_page(a, c, cache, job.src, job.dst, job.blocks, part, parts);
    if (first && cache == 0 && part == 0) {
      const int full = length(a, a.lens[job.parent]) >> a.shift;
      int32_t* to = a.table + job.row * a.stride;
      if (job.row != job.parent) {
        const int32_t* row = a.table + job.parent * a.stride;
        for (int j = threadIdx.x; j < full; j += kCopyThreads) {
          const int p = row[j];
          to[j] = p;
          if (in_pool(a, p)) atomicAdd(a.refs + p, 1);
        }
      } else if (threadIdx.x == 0) {
        atomicSub(a.refs + job.src, 1);
      }
      if (job.dst >= 0 && threadIdx.x == 0) to[full] = job.dst;
    }
  }
}

template <int S>
__global__ __launch_bounds__(kThreads) void compact_kernel(PagesArgs a, int32_t* held, int32_t* ws) {
  constexpr int kWindow = Free<S>::kWindow;
  __shared__ Scratch s;
  int32_t *rank = ws + 4, *dst = rank + a.n_pages, *src = dst + a.n_pages;
  Free<S> r{0};
  int n = 0, which = 0, all;
  for (int base = 0; base < a.n_pages; base += kWindow) {
    r = load_free<S>(a, base);
    scan_waves(s, which, count(base, r, [&](uint32_t id, bool free) { return id < (uint32_t)a.n_pages && !free; }), &all);
    which ^= 1;
    n += all;
  }
  const auto hole = [=](uint32_t id, bool free) { return id < (uint32_t)n && free; };
  const auto move = [&](uint32_t id, bool free) { return id >= (uint32_t)n && id < (uint32_t)a.n_pages && !free; };
  int holes = 0, moves = 0;                                    // of the windows before
  for (int base = 0; base < a.n_pages; base += kWindow) {
    if (a.n_pages > kWindow) r = load_free<S>(a, base);
    const int hole0 = holes + scan_waves(s, which, count(base, r, hole), &all);
    which ^= 1;
    holes += all;
    const int move0 = moves + scan_waves(s, which, count(base, r, move), &all);
    which ^= 1;
    moves += all;
    each(base, r, hole0, hole, [&](uint32_t id, bool yes, int k) {
      if (yes) dst[k] = id;
    });
    each(base, r, move0, move, [&](uint32_t id, bool yes, int k) {
      if (yes) src[k] = id;
      if (id >= (uint32_t)n && id < (uint32_t)a.n_pages) rank[id] = yes ? k : -1;
    });
  }
  if (threadIdx.x == 0) {
    ws[0] = moves;
    ws[1] = n;
    if (held) *held = n;
  }
}

__global__ __launch_bounds__(kCopyThreads) void compact_copy_kernel(PagesArgs a, const int32_t* ws, PageCopy c, int n_caches,
                                                                    bool first) {
  const int32_t *rank = ws + 4, *dst = rank + a.n_pages, *src = dst + a.n_pages;
  const int n = ws[1];
  const int64_t units = (int64_t)ws[0] * n_caches;
  const int parts = parts_of((int)min(units, (int64_t)gridDim.x));
  for (int64_t w = blockIdx.x; w < units * parts; w += gridDim.x) {
    const int64_t unit = w / parts;
    const int part = (int)(w % parts), k = (int)(unit / n_caches), cache = (int)(unit % n_caches);
    const int from = src[k], to = dst[k];
    if (c.heads[cache] > 0) copy_page(a, c, cache, from, to, 1 << (a.shift - 4), part, parts);
    if (first && cache == 0 && part == 0 && threadIdx.x == 0) {
      a.refs[to] = a.refs[from];
      a.refs[from] = 0;
    }
  }
  if (!first) return;
  for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
    const int have = pages(a, length(a, a.lens[b]));
    int32_t* row = a.table + b * a.stride;
    for (int j = threadIdx.x; j < have; j += kCopyThreads) {
      const int p = row[j];
      if (p < n || p >= a.n_pages) continue;
      const int k = rank[p];
      if (k >= 0) row[j] = dst[k];
    }
  }
}

// Pools of more than 32768 pages are gone through in windows of that many.
template <typename F>
void by_size(const PagesArgs& a, F f) {
  if (a.n_pages <= Free<1>::kWindow) f(std::integral_constant<int, 1>());
  else if (a.n_pages <= Free<4>::kWindow) f(std::integral_constant<int, 4>());
  else f(std::integral_constant<int, 8>());
}

}  // namespace

hipError_t launch_resize(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, hipStream_t s) {
  // 256 rows of up to 256 pages, half of which end: 48 us by one workgroup, ?? by two launches; one row: ?? and ??
  const bool many = (int64_t)a.seqs * a.per_seq > 8192;
  if (many) {
    const int x = a.per_seq < 1024 ? 1 : a.per_seq < 8192 ? a.per_seq / 1024 : 8;
    release_kernel<<<dim3((unsigned)x, (unsigned)a.seqs), dim3(256), 0, s>>>(a, new_lens);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  by_size(a, [&](auto steps) {
    resize_kernel<steps.value><<<dim3(1), dim3(kThreads), rows_lds(a.seqs), s>>>(a, new_lens, missing, many);
  });
  return hipGetLastError();
}

hipError_t launch_fork(const PagesArgs& a, const int32_t* from, int32_t* missing, void* ws, const PageCopy* c, int n_caches, int cus,
                       hipStream_t s) {
  int32_t* head = (int32_t*)ws;
  ForkJob* jobs = (ForkJob*)((uint8_t*)ws + kForkHead);
  by_size(a, [&](auto steps) {
    fork_kernel<steps.value><<<dim3(1), dim3(kThreads), rows_lds(a.seqs), s>>>(a, from, missing, head, jobs);
  });
  hipError_t e = hipGetLastError();
  for (int at = 0; e == hipSuccess && (at == 0 || at < n_caches); at += kCachesALaunch) {
    const int n = n_caches - at < kCachesALaunch ? n_caches - at : kCachesALaunch;
    fork_copy_kernel<<<dim3(4 * cus), dim3(kCopyThreads), 0, s>>>(a, head, jobs, c[at / kCachesALaunch], n > 0 ? n : 1, at == 0);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_compact(const PagesArgs& a, int32_t* held, int32_t* ws, const PageCopy* c, int n_caches, int cus, hipStream_t s) {
  by_size(a, [&](auto steps) { compact_kernel<steps.value><<<dim3(1), dim3(kThreads), 0, s>>>(a, held, ws); });
  hipError_t e = hipGetLastError();
  for (int at = 0; e == hipSuccess && (at == 0 || at < n_caches); at += kCachesALaunch) {
    const int n = n_caches - at < kCachesALaunch ? n_caches - at : kCachesALaunch;
    compact_copy_kernel<<<dim3(4 * cus), dim3(kCopyThreads), 0, s>>>(a, ws, c[at / kCachesALaunch], n > 0 ? n : 1, at == 0);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qmoe

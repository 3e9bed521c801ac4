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

#include "k_step.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct Scratch {
  int32_t wave[kWaves];
  int32_t total, granted;
};

// Sum of v over the threads before this one; all: over all of them.
__device__ __forceinline__ int scan(Scratch& s, int v, int* all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  __syncthreads();
  if (lane == 63) s.wave[wave] = sum;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int o = s.wave[i];
    before += i < wave ? o : 0;
    total += o;
  }
  *all = total;
  return before + sum - v;
}

// Goes through the ids of this wave's stretch of [0, n_pages) that `want` says yes to and returns their number.
// With kCall f(id, rank, yes) is called for every id of the stretch, rank being `first` and the number of yeses
// before it.
template <bool kCall, typename Want, typename F>
__device__ __forceinline__ int walk(const PagesArgs& a, int first, Want want, F f) {
  constexpr int kAhead = 4;                                    // loads in flight
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int steps = (a.n_pages + kThreads * 4 - 1) / (kThreads * 4);
  const uint64_t below = (1ull << lane) - 1;
  int rank = first;
  for (int i0 = 0; i0 < steps; i0 += kAhead) {
    i32x4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int id = ((wave * steps + i0 + u) * 64 + lane) * 4;
      v[u] = (i32x4){0, 0, 0, 0};
      if (i0 + u >= steps) continue;
      if (id + 4 <= a.n_pages) {
        v[u] = *(const i32x4*)(a.refs + id);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (id + c < a.n_pages) v[u][c] = a.refs[id + c];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int id = ((wave * steps + i0 + u) * 64 + lane) * 4;
      uint64_t yes[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) yes[c] = __ballot(i0 + u < steps && id + c < a.n_pages && want(id + c, v[u][c]));
      if (kCall) {
        int mine = rank;
#pragma unroll
        for (int c = 0; c < 4; ++c) mine += __popcll(yes[c] & below);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool is = (yes[c] >> lane) & 1;
          if (i0 + u < steps && id + c < a.n_pages) f(id + c, mine, is);
          mine += is;
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) rank += __popcll(yes[c]);
    }
  }
  return rank - first;
}

// The sum of every wave's v over the waves before this one; all: over all of them.
__device__ __forceinline__ int scan_waves(Scratch& s, int v, int* all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  __syncthreads();
  if (lane == 0) s.wave[wave] = v;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    before += i < wave ? s.wave[i] : 0;
    total += s.wave[i];
  }
  *all = total;
  return before;
}

// First index of a rising list (its sums, the own value included) whose sum is larger than v.
__device__ __forceinline__ int find(const int32_t* sums, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Grants the rows whose summed needs fit, and calls take(row, its which page, id) for their pages.
template <typename Take>
__device__ __forceinline__ void grant(const PagesArgs& a, Scratch& s, const int32_t* needs, int total, Take take) {
  if (threadIdx.x == 0) s.granted = 0;
  if (total == 0) {
    __syncthreads();
    return;
  }
  auto is_free = [](int, int refs) { return refs == 0; };
  const int mine = walk<false>(a, 0, is_free, [](int, int, bool) {});
  int free_pages;
  const int before = scan_waves(s, mine, &free_pages);
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    // (the last of the sums that fit)
    if (needs[b] <= free_pages && (b + 1 == a.seqs || needs[b + 1] > free_pages)) s.granted = needs[b];
  }
  __syncthreads();
  const int granted = s.granted;
  if (before < granted)
    walk<true>(a, before, is_free, [&](int id, int rank, bool yes) {
      if (!yes || rank >= granted) return;
      const int b = find(needs, a.seqs, rank);
      take(b, rank - (b ? needs[b - 1] : 0), id);
    });
}

__device__ __forceinline__ int length(const PagesArgs& a, int v) { return min(max(v, 0), a.per_seq << a.shift); }
__device__ __forceinline__ int pages(const PagesArgs& a, int len) { return (len + (1 << a.shift) - 1) >> a.shift; }
__device__ __forceinline__ bool in_pool(const PagesArgs& a, int p) { return p >= 0 && p < a.n_pages; }

__global__ __launch_bounds__(kThreads) void resize_kernel(PagesArgs a, const int32_t* new_lens, int32_t* missing) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  int32_t *drops = lds, *needs = lds + a.seqs;                 // sums over the rows up to each
  int drop_all = 0, need_all = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int drop = 0, need = 0;
    if (b < a.seqs) {
      const int old = length(a, a.lens[b]), to = new_lens[b];
      if (to >= 0) {
        const int d = pages(a, length(a, to)) - pages(a, old);
        drop = max(-d, 0);
        need = max(d, 0);
      }
    }
    int all;
    const int db = scan(s, drop, &all);
    if (b < a.seqs) drops[b] = drop_all + db + drop;
    drop_all += all;
    const int nb = scan(s, need, &all);
    if (b < a.seqs) needs[b] = need_all + nb + need;
    need_all += all;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < drop_all; i += kThreads) {
    const int b = find(drops, a.seqs, i);
    const int at = pages(a, length(a, new_lens[b])) + i - (b ? drops[b - 1] : 0);
    int32_t* e = a.table + b * a.stride + at;
    const int p = *e;
    *e = -1;
    if (in_pool(a, p)) atomicSub(a.refs + p, 1);
  }
  __threadfence();
  __syncthreads();
  grant(a, s, needs, need_all, [&](int b, int i, int id) {
    a.table[b * a.stride + pages(a, length(a, a.lens[b])) + i] = id;
    a.refs[id] = 1;
  });
  __syncthreads();
  const int granted = s.granted;
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    const int to = new_lens[b], need = needs[b] - (b ? needs[b - 1] : 0);
    if (to >= 0 && (need == 0 || needs[b] <= granted)) a.lens[b] = length(a, to);
  }
  if (missing && threadIdx.x == 0) *missing = need_all - granted;
}

__global__ __launch_bounds__(kThreads) void fork_kernel(PagesArgs a, const int32_t* from, int32_t* missing, int32_t* head,
                                                        ForkJob* jobs) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  int32_t *needs = lds, *where = lds + a.seqs;                 // sums of needs; a row's job (of those that need a page)
  int need_all = 0, job_all = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    ForkJob job{b, -1, -1, -1, 0};
    if (b < a.seqs) {
      const int p = from[b];
      if (p >= 0 && p < a.seqs) {
        const int len = length(a, a.lens[p]), rest = len & ((1 << a.shift) - 1);
        if (len > 0 && (p == b ? rest > 0 : length(a, a.lens[b]) == 0)) {
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
    const int nb = scan(s, need, &all);
    if (b < a.seqs) needs[b] = need_all + nb + need;
    need_all += all;
    const int at = job_all + scan(s, job.parent >= 0, &all);
    job_all += all;
    if (job.parent >= 0) jobs[at] = job;
    if (b < a.seqs) where[b] = job.parent >= 0 ? at : -1;
  }
  __threadfence();
  __syncthreads();
  grant(a, s, needs, need_all, [&](int b, int, int id) {
    jobs[where[b]].dst = id;
    a.refs[id] = 1;
  });
  __syncthreads();
  const int granted = s.granted;
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    if (where[b] < 0) continue;
    const int need = needs[b] - (b ? needs[b - 1] : 0);
    if (need && needs[b] > granted) jobs[where[b]].parent = -1;
    else if (from[b] != b) a.lens[b] = length(a, a.lens[from[b]]);
  }
  if (threadIdx.x == 0) {
    *head = job_all;
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

__global__ __launch_bounds__(kThreads) void compact_kernel(PagesArgs a, int32_t* held, int32_t* ws) {
  __shared__ Scratch s;
  int32_t *rank = ws + 4, *dst = rank + a.n_pages, *src = dst + a.n_pages;
  auto none = [](int, int, bool) {};
  int n, holes, moves;
  scan_waves(s, walk<false>(a, 0, [](int, int refs) { return refs != 0; }, none), &n);
  auto hole = [=](int id, int refs) { return id < n && refs == 0; };
  auto move = [=](int id, int refs) { return id >= n && refs != 0; };
  const int hole0 = scan_waves(s, walk<false>(a, 0, hole, none), &holes);
  const int move0 = scan_waves(s, walk<false>(a, 0, move, none), &moves);
  walk<true>(a, hole0, hole, [&](int id, int k, bool yes) {
    if (yes) dst[k] = id;
  });
  walk<true>(a, move0, move, [&](int id, int k, bool yes) {
    if (yes) src[k] = id;
    if (id >= n) rank[id] = yes ? k : -1;
  });
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

}  // namespace

hipError_t launch_resize(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, hipStream_t s) {
  resize_kernel<<<dim3(1), dim3(kThreads), (size_t)a.seqs * 8, s>>>(a, new_lens, missing);
  return hipGetLastError();
}

hipError_t launch_fork(const PagesArgs& a, const int32_t* from, int32_t* missing, void* ws, const PageCopy* c, int n_caches, int cus,
                       hipStream_t s) {
  int32_t* head = (int32_t*)ws;
  ForkJob* jobs = (ForkJob*)((uint8_t*)ws + kForkHead);
  fork_kernel<<<dim3(1), dim3(kThreads), (size_t)a.seqs * 8, s>>>(a, from, missing, head, jobs);
  hipError_t e = hipGetLastError();
  for (int at = 0; e == hipSuccess && (at == 0 || at < n_caches); at += kCachesALaunch) {
    const int n = n_caches - at < kCachesALaunch ? n_caches - at : kCachesALaunch;
    fork_copy_kernel<<<dim3(4 * cus), dim3(kCopyThreads), 0, s>>>(a, head, jobs, c[at / kCachesALaunch], n > 0 ? n : 1, at == 0);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_compact(const PagesArgs& a, int32_t* held, int32_t* ws, const PageCopy* c, int n_caches, int cus, hipStream_t s) {
  compact_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(a, held, ws);
  hipError_t e = hipGetLastError();
  for (int at = 0; e == hipSuccess && (at == 0 || at < n_caches); at += kCachesALaunch) {
    const int n = n_caches - at < kCachesALaunch ? n_caches - at : kCachesALaunch;
    compact_copy_kernel<<<dim3(4 * cus), dim3(kCopyThreads), 0, s>>>(a, ws, c[at / kCachesALaunch], n > 0 ? n : 1, at == 0);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qmoe

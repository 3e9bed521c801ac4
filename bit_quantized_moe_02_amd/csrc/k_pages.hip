// Pages of a key/value cache kept on the GPU (moe_kv_resize, moe_kv_fork,
// moe_kv_compact).
//
// What has to be decided is small (lengths, one count of holders a page) and
// goes one after the other (rows take free pages in order), so one workgroup
// decides it.  Counts of a pool are looked through once, 64 ids to a word of
// bits; sums over rows and words give each row its place among the free pages, and the
// threads that own the words list these in LDS for the rows.  There is no list of
// free pages in memory: the lowest free ids are taken, whatever order they were
// given back in, so that results do not depend on the order of atomics.  Page
// contents are copied by a second launch over the whole card.
//
// Latency bounds the decisions: a launch is 2 us, each load that another one
// needs about 0.7.  Of a call on the GPU: a row that grows by a token 2.6 us, 64 rows of
// 16 pages 2.6 with nothing to do, 5 with a page to take each; 256 rows of a pool of 24000 pages 5.2, growing by 70 pages each
// 9; the fork's decision 3.5, the compaction's 3.2 (2048 pages 4.9).  Bytes bound the copies: 849 MB read and written
// in 175 us (4.8 TB/s), 71 MB in 14.4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "k_step.h"
#include "lds_limit.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// v with the (uniform) word in one lane: there is no builtin for the instruction.
extern "C" __device__ uint32_t write_lane(uint32_t word, uint32_t lane, uint32_t v) __asm("llvm.amdgcn.writelane.i32");

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct Scratch {
  int32_t wave[2][kWaves];
};

// Sums over the lanes up to this one, by moves between registers.
__device__ __forceinline__ int scan_row(int v) {               // of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  return v;
}
__device__ __forceinline__ int scan_wave(int v) {
  v = scan_row(v);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // the last of the row before, to the second and fourth
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // the last of the first half, to the second
  return v;
}

// Sums of v over the threads before this one and over all of them.  `which` alternates between calls, so that one barrier
// a call is enough.
__device__ __forceinline__ int scan(Scratch& s, int& which, int v, int* all) {
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int sum = scan_wave(v);
  if (lane == 63) s.wave[which][wave] = sum;
  __syncthreads();
  const int waves = scan_row(s.wave[which][lane % kWaves]);    // (16 waves)
  const int before = wave ? __builtin_amdgcn_readlane(waves, wave - 1) : 0;
  which ^= 1;
  *all = __builtin_amdgcn_readlane(waves, kWaves - 1);
  return before + sum - v;
}

// Which ids of a window of 4096 * S are free: words of 64 ids, bit by bit.
template <int S>
struct Free {
  static constexpr int kWords = 64 * S, kWindow = 64 * kWords;
  uint64_t word[kWords];
};

// Of 64 ids from `id` on, those below n.
__device__ __forceinline__ uint64_t ids_below(uint32_t id, uint32_t n) {
  return id >= n ? 0 : n - id >= 64 ? ~0ull : (1ull << (n - id)) - 1;
}

// The window's words (ids past the pool are not free).  A wave's load is a word's 64 ids, a lane keeps one of its wave's
// words: a comparison and two moves a word.  (Four ids a lane, put together by 16 lanes, took 4 us of a window of 65536.)
// kFresh: not from the first-level cache, which does not see the atomics.
template <bool kFresh = false, int S>
__device__ __forceinline__ void load_free(const PagesArgs& a, int base, Free<S>& f) {
  constexpr int kLoads = Free<S>::kWords / kWaves, kAtOnce = kLoads < 16 ? kLoads : 16;
  const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // (past the end of it a buffer reads as zeros)
  const __amdgpu_buffer_rsrc_t refs = __builtin_amdgcn_make_buffer_rsrc(a.refs, 0, (int)((uint32_t)a.n_pages * 4), 0x00027000);
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i0 = 0; i0 < kLoads; i0 += kAtOnce) {
    if ((uint32_t)base + i0 * kWaves * 64 >= (uint32_t)a.n_pages) break;
    int v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      v[i] = __builtin_amdgcn_raw_buffer_load_b32(refs, ((uint32_t)base + ((i0 + i) * kWaves + wave) * 64 + lane) * 4, 0, kFresh ? 16 : 0);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint64_t w = __builtin_amdgcn_ballot_w64(v[i] == 0);
      lo = write_lane((uint32_t)w, i0 + i, lo);
      hi = write_lane((uint32_t)(w >> 32), i0 + i, hi);
    }
  }
  const int at = lane * kWaves + wave;
  if (lane < kLoads) f.word[at] = ((uint64_t)hi << 32 | lo) & ids_below((uint32_t)base + at * 64, a.n_pages);
}

// A number that is the same in all lanes, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// Of a (uniform) word's ids a lane takes one: how many set ones come before it.
__device__ __forceinline__ int set_before(uint64_t w) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(w >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)w, 0));
}

// Numbers of LDS: sums of the rows' needs and another number a row; a list of free pages, as many as there is room for.
struct Rows {
  int32_t *needs, *x, *list;
  int most;
  __device__ Rows(int32_t* lds, int seqs, int n) : needs(lds), x(needs + seqs), list(x + seqs), most(n) {}
};
// (one workgroup has all of LDS to itself: 160 KB less what is declared, at most)
constexpr int kDeclared = 16384;
inline int list_of(const PagesArgs& a) { return a.n_pages < 36864 - 2 * a.seqs ? a.n_pages : 36864 - 2 * a.seqs; }
inline size_t rows_lds(const PagesArgs& a) { return ((size_t)list_of(a) + 2 * (size_t)a.seqs) * 4; }

// Gives the rows whose summed needs fit the lowest free pages, in order: give(first, n) is called with pages of ranks
// first .. first + n - 1 in the list.  Returns how many pages the rows were given.  f: the words of the first window.
template <int S, typename Give>
__device__ __forceinline__ int grant(const PagesArgs& a, Scratch& s, int& which, const Rows& rows, int total, Free<S>& f, Give give) {
  constexpr int kWindow = Free<S>::kWindow;
  if (total == 0) return 0;
  __shared__ int32_t fits;
  // A thread has one word: its free pages, and the rank of the first of them.
  uint64_t bits = 0;
  int rank = 0;
  auto ranks = [&](int passed) {
    bits = threadIdx.x < Free<S>::kWords ? f.word[threadIdx.x] : 0;
    int all;
    rank = passed + scan(s, which, __popcll(bits), &all);
    return all;
  };
  int free_pages = 0;
  for (int base = 0; base < a.n_pages && free_pages < total; base += kWindow) {
    if (base) {
      __syncthreads();
      load_free<true>(a, base, f);
      __syncthreads();
    }
    free_pages += ranks(free_pages);
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
  int passed = 0;                                             // free pages of the windows before
  // (The windows are looked through once more: should another call on the pool have taken pages in between, there are fewer
  // than were counted, and the pool's end ends it.)
  for (int base = 0; passed < granted && base < a.n_pages; base += kWindow) {
    int all = free_pages;
    if (a.n_pages > kWindow) {
      __syncthreads();
      load_free<true>(a, base, f);
      __syncthreads();
      all = ranks(passed);
    }
    const int last = min(granted, passed + all);
    for (int first = passed; first < last; first += rows.most) {
      const int end = min(first + rows.most, last);
      for (; bits && rank < end; ++rank, bits &= bits - 1) rows.list[rank - first] = base + threadIdx.x * 64 + __builtin_ctzll(bits);
      __syncthreads();
      give(first, end - first);
      if (end < granted) __syncthreads();                     // (the list is written again)
    }
    passed += all;
  }
  return min(granted, passed);
}

__device__ __forceinline__ int length(const PagesArgs& a, int v) { return min(max(v, 0), a.per_seq << a.shift); }
__device__ __forceinline__ int pages(const PagesArgs& a, int len) { return (len + (1 << a.shift) - 1) >> a.shift; }
__device__ __forceinline__ bool in_pool(const PagesArgs& a, int p) { return p >= 0 && p < a.n_pages; }

// Entries from..to-1 of a row given back, by `lanes` threads of which this is number `lane`.
template <int kScope>
__device__ __forceinline__ void release(const PagesArgs& a, int b, int from, int to, int lane, int lanes) {
  int32_t* row = a.table + b * a.stride;
#pragma unroll 4
  for (int j = from + lane; j < to; j += lanes) {
    const int p = row[j];
    row[j] = -1;
    if (in_pool(a, p)) __hip_atomic_fetch_sub(a.refs + p, 1, __ATOMIC_RELAXED, kScope);
  }
}

// The rows' pages given back by the whole card, where there may be many: the counts of 16000 take one compute unit 8 us.
__global__ __launch_bounds__(256) void release_kernel(PagesArgs a, const int32_t* new_lens) {
  const int b = blockIdx.y, old = a.lens[b], to = new_lens[b];
  if (to < 0) return;
  release<__HIP_MEMORY_SCOPE_AGENT>(a, b, pages(a, length(a, to)), pages(a, length(a, old)), blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

template <int S>
__global__ __launch_bounds__(kThreads) void resize_kernel(PagesArgs a, const int32_t* new_lens, int32_t* missing, bool released, int list) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  __shared__ Free<S> f;
  const Rows rows(lds, a.seqs, list);                                // x: pages held
  int need_all = 0, which = 0;
  bool drops = false;
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int old = 0, to = -1;
    if (b < a.seqs) {
      old = a.lens[b];
      to = new_lens[b];
    }
    if (b0 == 0) load_free(a, 0, f);                           // (for the case that none is given back)
    const int have = pages(a, length(a, old)), want = to < 0 ? have : pages(a, length(a, to));
    drops |= want < have;
    int all;
    const int before = scan(s, which, max(want - have, 0), &all);
    if (b < a.seqs) {
      rows.x[b] = have;
      rows.needs[b] = need_all + before + max(want - have, 0);
    }
    need_all += all;
  }
  // 16 threads a row, or as many as there are for fewer than 64 rows
  int lanes = 16;
  while (lanes < kThreads && lanes * a.seqs < kThreads) lanes *= 2;
  const int group = threadIdx.x / lanes, groups = kThreads / lanes, lane = threadIdx.x % lanes;
  if (__syncthreads_or(drops && !released)) {
    for (int b = group; b < a.seqs; b += groups) {
      const int to = new_lens[b];
      if (to >= 0) release<__HIP_MEMORY_SCOPE_WORKGROUP>(a, b, pages(a, length(a, to)), rows.x[b], lane, lanes);
    }
    if (need_all) {
      // (the counts are this workgroup's alone: its atomics done, in the second-level cache, is enough)
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      load_free<true>(a, 0, f);
      __syncthreads();
    }
  }
  const int granted = grant(a, s, which, rows, need_all, f, [&](int first, int n) {
    for (int b = group; b < a.seqs; b += groups) {
      const int end = rows.needs[b], begin = b ? rows.needs[b - 1] : 0;
      if (end <= first || begin >= first + n) continue;
      int32_t* to = a.table + b * a.stride + rows.x[b] - begin;
#pragma unroll 4
      for (int i = max(begin, first) + lane; i < min(end, first + n); i += lanes) {
        const int p = rows.list[i - first];
        to[i] = p;
        a.refs[p] = 1;
      }
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
                                                        ForkJob* jobs, int list) {
  extern __shared__ int32_t lds[];
  __shared__ Scratch s;
  __shared__ Free<S> f;
  const Rows rows(lds, a.seqs, list);                                // x: the row's job (-1: none)
  int sums = 0, which = 0;                                     // jobs, and in the upper half needs, of the rows before
  for (int b0 = 0; b0 < a.seqs; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0, p = -1, own = 0;
    ForkJob job{b, -1, -1, -1, 0};
    if (b < a.seqs) {
      p = from[b];
      own = length(a, a.lens[b]);
    }
    if (b0 == 0) load_free(a, 0, f);
    if (p >= 0 && p < a.seqs) {
      const int len = length(a, a.lens[p]), rest = len & ((1 << a.shift) - 1);
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
    int all;
    const int before = sums + scan(s, which, (job.parent >= 0) | need << 16, &all);
    sums += all;
    if (job.parent >= 0) jobs[before & 0xFFFF] = job;
    if (b < a.seqs) {
      rows.needs[b] = (before >> 16) + need;
      rows.x[b] = job.parent >= 0 ? before & 0xFFFF : -1;
    }
  }
  const int need_all = sums >> 16;
  __syncthreads();
  const int granted = grant(a, s, which, rows, need_all, f, [&](int first, int n) {
    for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
      const int end = rows.needs[b], begin = b ? rows.needs[b - 1] : 0;
      if (end > begin && begin >= first && begin < first + n) {
        const int p = rows.list[begin - first];
        jobs[rows.x[b]].dst = p;
        a.refs[p] = 1;
      }
    }
  });
  for (int b = threadIdx.x; b < a.seqs; b += kThreads) {
    if (rows.x[b] < 0) continue;
    const int end = rows.needs[b], need = end - (b ? rows.needs[b - 1] : 0), p = from[b];
    if (need && end > granted) jobs[rows.x[b]].parent = -1;
    else if (p != b) a.lens[b] = length(a, a.lens[p]);         // (a parent's own length does not change here)
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
  constexpr int kWindow = Free<S>::kWindow, kWords = Free<S>::kWords;
  __shared__ Scratch s;
  __shared__ Free<S> f;
  __shared__ int32_t filled[kWords], moving[kWords];           // ranks of a word's first hole and moving page
  int32_t *rank = ws + 4, *dst = rank + a.n_pages, *src = dst + a.n_pages;
  const int t = threadIdx.x, lane = t % 64, wave = uniform(t / 64);
  int n = a.n_pages, which = 0, all;
  for (int base = 0; base < a.n_pages; base += kWindow) {
    load_free(a, base, f);
    __syncthreads();
    scan(s, which, t < kWords ? __popcll(f.word[t]) : 0, &all);
    n -= all;
    if (a.n_pages > kWindow) __syncthreads();                  // (the words are written again)
  }
  int holes = 0, moves = 0;                                    // of the windows before
  for (int base = 0; base < a.n_pages; base += kWindow) {
    if (a.n_pages > kWindow) {
      load_free(a, base, f);
      __syncthreads();
    }
    uint64_t hole = 0, move = 0;
    if (t < kWords) {
      const uint32_t id = base + t * 64;
      hole = f.word[t] & ids_below(id, n);
      move = ~f.word[t] & ~ids_below(id, n) & ids_below(id, a.n_pages);
    }
    const int k = holes + scan(s, which, __popcll(hole), &all);
    holes += all;
    const int l = moves + scan(s, which, __popcll(move), &all);
    moves += all;
    if (t < kWords) {
      filled[t] = k;
      moving[t] = l;
    }
    __syncthreads();
    for (int i = wave; i < kWords; i += kWaves) {
      const uint32_t id = base + i * 64, p = id + lane;
      if (id >= (uint32_t)a.n_pages) break;
      const uint64_t w = uniform(f.word[i]), low = ids_below(id, n), hole = w & low, move = ~w & ~low & ids_below(id, a.n_pages);
      if (__builtin_amdgcn_inverse_ballot_w64(hole)) dst[filled[i] + set_before(hole)] = p;
      const bool moved = __builtin_amdgcn_inverse_ballot_w64(move);
      const int number = moving[i] + set_before(move);
      if (moved) src[number] = p;
      if (p >= (uint32_t)n && p < (uint32_t)a.n_pages) rank[p] = moved ? number : -1;
    }
    __syncthreads();
  }
  if (t == 0) {
    ws[0] = min(moves, holes);                                 // (the same, unless another call changed the pool meanwhile)
    ws[1] = n;
    if (held) *held = n;
  }
}

__global__ __launch_bounds__(kCopyThreads) void compact_copy_kernel(PagesArgs a, const int32_t* ws, PageCopy c, int n_caches,
                                                                    bool first) {
  const int32_t *rank = ws + 4, *dst = rank + a.n_pages, *src = dst + a.n_pages;
  const int n = ws[1], moves = ws[0];
  const int64_t units = (int64_t)moves * n_caches;
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
      if (k >= 0 && k < moves) row[j] = dst[k];
    }
  }
}

// Pools of more than 65536 pages are gone through in windows of that many; up to 4096 in one load of each wave's, which saves
// 0.3 us a call (64 rows of a pool of 2000 2.6 for 2.9; windows of 16384 saved nothing).
template <typename F>
void by_size(const PagesArgs& a, F f) {
  if (a.n_pages <= Free<1>::kWindow) f(std::integral_constant<int, 1>());
  else f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_resize(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, hipStream_t s) {
  // The launch costs 3.4 us where there is nothing to give back.  Pairs of calls that take all pages and give back all but
  // a few: 256 rows of 32 pages 15.3 us without it, 15.3 with it, of 64 20.7 and 17.2, of 128 30 and 20; by a token each of 64 14.8 and
  // 16.0, of 128 15.9 and 17.1.
  const bool many = (int64_t)a.seqs * a.per_seq > 16384;
  if (many) {
    const int x = a.per_seq < 1024 ? 1 : a.per_seq < 8192 ? a.per_seq / 1024 : 8;
    release_kernel<<<dim3((unsigned)x, (unsigned)a.seqs), dim3(256), 0, s>>>(a, new_lens);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipError_t e = hipSuccess;
  by_size(a, [&](auto steps) {
    const auto kernel = resize_kernel<steps.value>;
    if (rows_lds(a) > 32768) e = raise_dyn_lds((const void*)kernel, kDeclared);
    if (e == hipSuccess) kernel<<<dim3(1), dim3(kThreads), rows_lds(a), s>>>(a, new_lens, missing, many, list_of(a));
  });
  return e == hipSuccess ? hipGetLastError() : e;
}

hipError_t launch_fork(const PagesArgs& a, const int32_t* from, int32_t* missing, void* ws, const PageCopy* c, int n_caches, int cus,
                       hipStream_t s) {
  int32_t* head = (int32_t*)ws;
  ForkJob* jobs = (ForkJob*)((uint8_t*)ws + kForkHead);
  hipError_t e = hipSuccess;
  by_size(a, [&](auto steps) {
    const auto kernel = fork_kernel<steps.value>;
    if (rows_lds(a) > 32768) e = raise_dyn_lds((const void*)kernel, kDeclared);
    if (e == hipSuccess) kernel<<<dim3(1), dim3(kThreads), rows_lds(a), s>>>(a, from, missing, head, jobs, list_of(a));
  });
  if (e == hipSuccess) e = hipGetLastError();
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

// Pages of the cache: fork, resize, compact, copy.
//
// The state is refs [num_pages] (how many table entries hold a page; 0: the
// page is free), table [rows][max_pages] and lens [rows].  A call takes free
// pages lowest first, in the order of its rows, so its result is determined
// by its arguments.  Two launches: one workgroup plans (checks, counts,
// finds the free pages) and writes what is to be done to the workspace; then
// the chip copies pages and writes tables.  A plan that cannot be carried out
// changes nothing.
//
// The whole-chip kernel is bound by HBM (a page is layers * kv_heads *
// (128 D + 32) bytes, read and written); the plan by the latency of its few
// dependent rounds, which is why it only scans refs as far as it needs.
// Measured with 600 pages of 2 MB: plan of a fork into 8 rows 5.2 us and 7.0
// us to carry it out, of a resize 6.6 and 5.0, of a compaction 4.7 and, with
// 143 moves, 123 us (4.9 TB/s).
#pragma once

#include "kv_common.hpp"

namespace bq {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
// Bytes that a workgroup moves at a time: 16 a thread.  A layer's K or V of a
// page is whole units of this.
constexpr int kCopyUnit = kCopyThreads * 16;

struct KvPool {
  uint8_t *k, *v;
  float *ks, *vs;
  int layers, num_pages;
  int64_t page_bytes;  // of one layer's K or V: kv_heads * 64 * D
  int page_scales;     // floats of one layer: kv_heads * 4
};

// Workspace: go, number of copies, then the arrays.
struct KvPlan {
  int* head;   // [0] 1: carry it out, [1] copies
  int* src;    // [num_pages] pages to copy from
  int* dst;    // [num_pages] to
  int* take;   // [num_pages] free pages in the order in which they are taken, or the new id of each page
  int* row;    // [2 * rows] of each row: first of its taken pages, and its length or whether its last page is copied
};
constexpr int kPlanHead = 16;
inline size_t kv_plan_ints(int num_pages, int rows) { return kPlanHead + 3 * (size_t)num_pages + 2 * (size_t)rows; }

struct KvPagesParams {
  KvPool pool;
  KvPlan plan;
  int *table, *lens, *refs, *status;
  const int *a, *b;  // fork: src, dst; resize: want; copy: src, dst
  int rows, max_pages, n;
};

// refs are changed by atomics of this launch: read where those are performed
__device__ __forceinline__ int kv_ref(const int* refs, int p) {
  return __hip_atomic_load(refs + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive prefix of one value a thread over the workgroup, and the total.
__device__ __forceinline__ int plan_scan(int v, int& total) {
  __shared__ int waves[kPlanThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(s, o, 64);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    before += w < wave ? waves[w] : 0;
    total += waves[w];
  }
  return before + s - v;
}

// The first `need` free pages, in order, to take[]; how many there are.
__device__ __forceinline__ int plan_take(const KvPagesParams& p, int need) {
  int found = 0;
  for (int base = 0; base < p.pool.num_pages && found < need; base += kPlanThreads) {
    const int id = base + (int)threadIdx.x;
    const int is = id < p.pool.num_pages && kv_ref(p.refs, id) == 0;
    int total;
    const int at = found + plan_scan(is, total);
    if (is && at < need) p.plan.take[at] = id;
    found += total;
  }
  return found;
}

__device__ __forceinline__ void plan_say(const KvPagesParams& p, int go, int copies, int told) {
  if (threadIdx.x == 0) {
    p.plan.head[0] = go;
    p.plan.head[1] = go ? copies : 0;
    p.status[0] = told;
    p.status[1] = go ? copies : 0;
  }
}

__global__ __launch_bounds__(kPlanThreads) void kv_fork_plan_kernel(KvPagesParams p) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  for (int i = (int)threadIdx.x; i < p.rows; i += kPlanThreads) p.plan.row[p.rows + i] = 0;
  __syncthreads();
  // row[rows + dst]: how often a row is a destination
  int need = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + (int)threadIdx.x;
    int tail = 0;
    if (i < p.n) {
      const int src = p.a[i], dst = p.b[i];
      bool ok = (unsigned)src < (unsigned)p.rows && (unsigned)dst < (unsigned)p.rows && src != dst;
      if (ok) {
        const int len = p.lens[src];
        ok = p.lens[dst] == 0 && len >= 0 && len <= p.max_pages * kKvPage && atomicAdd(&p.plan.row[p.rows + dst], 1) == 0;
        tail = ok && len % kKvPage != 0;
        if (tail) ok = (unsigned)p.table[(int64_t)src * p.max_pages + len / kKvPage] < (unsigned)p.pool.num_pages;
      }
      if (!ok) atomicAdd(&bad, 1);
    }
    int total;
    const int at = need + plan_scan(tail, total);
    if (i < p.n) p.plan.row[i] = at;  // n <= rows
    need += total;
  }
  __syncthreads();
  if (bad) return plan_say(p, 0, 0, -1);
  const int found = plan_take(p, need);
  if (found < need) return plan_say(p, 0, 0, need - found);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < p.n; i += kPlanThreads) {
    const int src = p.a[i], len = p.lens[src], at = p.plan.row[i];
    if (len % kKvPage != 0) {
      p.plan.src[at] = p.table[(int64_t)src * p.max_pages + len / kKvPage];
      p.plan.dst[at] = p.plan.take[at];
    }
  }
  __syncthreads();
  // from here on row[rows + i] is the length of fork i
  for (int i = (int)threadIdx.x; i < p.n; i += kPlanThreads) p.plan.row[p.rows + i] = p.lens[p.a[i]];
  plan_say(p, 1, need, 0);
}

__global__ __launch_bounds__(kPlanThreads) void kv_resize_plan_kernel(KvPagesParams p) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = (int)threadIdx.x; i < p.rows; i += kPlanThreads) {
    const int len = p.lens[i], want = p.a[i];
    if (want < -1 || want > p.max_pages * kKvPage || len < 0 || len > p.max_pages * kKvPage) atomicAdd(&bad, 1);
  }
  __syncthreads();
  if (bad) return plan_say(p, 0, 0, -1);
  // pages past the wanted lengths are let go (taken back below if the call
  // cannot be carried out); a wave takes a row
  const auto drop = [&](int by) {
    for (int i = wave; i < p.rows; i += kPlanThreads / 64) {
      const int len = p.lens[i], want = p.a[i] < 0 ? len : p.a[i];
      const int have = (len + kKvPage - 1) / kKvPage;
      for (int c = (want + kKvPage - 1) / kKvPage + lane; c < have; c += 64) {
        const int id = p.table[(int64_t)i * p.max_pages + c];
        if ((unsigned)id < (unsigned)p.pool.num_pages)
          __hip_atomic_fetch_add(&p.refs[id], by, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    // performed before the reads after the barrier
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  drop(-1);
  int need = 0, copies = 0;
  for (int base = 0; base < p.rows; base += kPlanThreads) {
    const int i = base + (int)threadIdx.x;
    int count = 0, split = 0;
    if (i < p.rows) {
      const int len = p.lens[i], want = p.a[i] < 0 ? len : p.a[i];
      const int have = (len + kKvPage - 1) / kKvPage, need_i = (want + kKvPage - 1) / kKvPage;
      if (want < len && want % kKvPage != 0) {
        const int id = p.table[(int64_t)i * p.max_pages + need_i - 1];
        split = (unsigned)id < (unsigned)p.pool.num_pages && kv_ref(p.refs, id) > 1;
      }
      count = max(need_i - have, 0) + split;
    }
    int total, total_copies;
    const int at = need + plan_scan(count, total);
    const int copy_at = copies + plan_scan(split, total_copies);
    if (i < p.rows) {
      p.plan.row[i] = at;
      p.plan.row[p.rows + i] = split ? copy_at : -1;
    }
    need += total;
    copies += total_copies;
  }
  const int found = plan_take(p, need);
  __syncthreads();
  if (found < need) {
    drop(1);
    return plan_say(p, 0, 0, need - found);
  }
  for (int i = (int)threadIdx.x; i < p.rows; i += kPlanThreads) {
    const int copy_at = p.plan.row[p.rows + i];
    if (copy_at >= 0) {
      p.plan.src[copy_at] = p.table[(int64_t)i * p.max_pages + (p.a[i] + kKvPage - 1) / kKvPage - 1];
      p.plan.dst[copy_at] = p.plan.take[p.plan.row[i]];
    }
  }
  plan_say(p, 1, copies, 0);
}

__global__ __launch_bounds__(kPlanThreads) void kv_compact_plan_kernel(KvPagesParams p) {
  int live = 0;
  for (int base = 0; base < p.pool.num_pages; base += kPlanThreads) {
    const int id = base + (int)threadIdx.x;
    int total;
    plan_scan(id < p.pool.num_pages && p.refs[id] > 0, total);
    live += total;
  }
  int up = 0, down = 0;  // live pages from `live` on, free pages below it
  for (int base = 0; base < p.pool.num_pages; base += kPlanThreads) {
    const int id = base + (int)threadIdx.x;
    const bool in = id < p.pool.num_pages, is = in && p.refs[id] > 0;
    int n_up, n_down;
    const int at_up = up + plan_scan(is && id >= live, n_up);
    const int at_down = down + plan_scan(in && !is && id < live, n_down);
    if (is && id >= live) p.plan.src[at_up] = id;
    if (in && !is && id < live) p.plan.dst[at_down] = id;
    if (in && !is && id >= live) p.plan.take[id] = -1;
    up += n_up;
    down += n_down;
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < up; i += kPlanThreads) p.plan.take[p.plan.src[i]] = p.plan.dst[i];
  if (threadIdx.x == 0) p.plan.head[2] = live;
  plan_say(p, 1, up, 0);
}

// Copies of pages over all layers.  The grid's x is a layer's K or V, its y a
// unit of kCopyUnit bytes of every (gridDim.y / units)-th pair: workgroups go
// to the eight XCDs in turn, so with x first each XCD translates the addresses
// of its own layers only.  Measured, pages of 2 MB in 16 layers: 8 pages 7.3
// us, 200 pages 168 us (5.0 TB/s read and written); with two, four or eight 16-byte
// loads a thread 19.2, 19.3, 10.4 and 173, 173, 204 us.  Ids out of range (the
// caller's own lists) are skipped.
__device__ __forceinline__ void copy_pages(const KvPool& c, const int* src, const int* dst, int count) {
  const unsigned units = (unsigned)(c.page_bytes / kCopyUnit);
  const unsigned first = blockIdx.y / units, unit = blockIdx.y - first * units, step = gridDim.y / units;
  const int which = (int)blockIdx.x & 1, layer = (int)blockIdx.x >> 1;
  uint8_t* codes = which ? c.v : c.k;
  float* scales = which ? c.vs : c.ks;
  const int64_t at = (int64_t)unit * kCopyUnit + threadIdx.x * 16;
  for (unsigned pair = first; pair < (unsigned)count; pair += step) {
    const int from = src[pair], to = dst[pair];
    if ((unsigned)from >= (unsigned)c.num_pages || (unsigned)to >= (unsigned)c.num_pages || from == to) continue;
    const int64_t fp = (int64_t)layer * c.num_pages + from, tp = (int64_t)layer * c.num_pages + to;
    const uint8_t* f = codes + fp * c.page_bytes + at;
    uint8_t* t = codes + tp * c.page_bytes + at;
    *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(f);
    if (unit == 0)
      for (int e = (int)threadIdx.x; e < c.page_scales; e += kCopyThreads)
        scales[tp * c.page_scales + e] = scales[fp * c.page_scales + e];
  }
}

__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(KvPagesParams p) {
  copy_pages(p.pool, p.a, p.b, p.n);
}

__global__ __launch_bounds__(kCopyThreads) void kv_fork_kernel(KvPagesParams p) {
  if (!p.plan.head[0]) return;
  const int wg = (int)(blockIdx.y * gridDim.x + blockIdx.x), wgs = (int)(gridDim.x * gridDim.y);
  for (int i = wg; i < p.n; i += wgs) {
    const int src = p.a[i], dst = p.b[i], len = p.plan.row[p.rows + i], full = len / kKvPage;
    const int tail = len % kKvPage != 0;
    for (int c = (int)threadIdx.x; c < p.max_pages; c += kCopyThreads) {
      int id = -1;
      if (c < full) {
        id = p.table[(int64_t)src * p.max_pages + c];
        if ((unsigned)id < (unsigned)p.pool.num_pages) atomicAdd(&p.refs[id], 1);
      } else if (tail && c == full) {
        id = p.plan.take[p.plan.row[i]];
        p.refs[id] = 1;
      }
      p.table[(int64_t)dst * p.max_pages + c] = id;
    }
    if (threadIdx.x == 0) p.lens[dst] = len;
  }
  copy_pages(p.pool, p.plan.src, p.plan.dst, p.plan.head[1]);
}

__global__ __launch_bounds__(kCopyThreads) void kv_resize_kernel(KvPagesParams p) {
  if (!p.plan.head[0]) return;
  const int wg = (int)(blockIdx.y * gridDim.x + blockIdx.x), wgs = (int)(gridDim.x * gridDim.y);
  for (int i = wg; i < p.rows; i += wgs) {
    const int len = p.lens[i], want = p.a[i] < 0 ? len : p.a[i];
    const int have = (len + kKvPage - 1) / kKvPage, need = (want + kKvPage - 1) / kKvPage;
    int* row = p.table + (int64_t)i * p.max_pages;
    const int first = p.plan.row[i];
    for (int c = min(have, need) + (int)threadIdx.x; c < max(have, need); c += kCopyThreads) {
      int id = -1;
      if (c >= have) {
        id = p.plan.take[first + c - have];
        p.refs[id] = 1;
      }
      row[c] = id;
    }
    __syncthreads();  // every thread has read lens[i]
    if (threadIdx.x == 0) {
      const int copy = p.plan.row[p.rows + i];
      if (copy >= 0) {
        const int id = p.plan.dst[copy];
        row[need - 1] = id;
        p.refs[id] = 1;
        atomicAdd(&p.refs[p.plan.src[copy]], -1);
      }
      p.lens[i] = want;
    }
  }
  copy_pages(p.pool, p.plan.src, p.plan.dst, p.plan.head[1]);
}

__global__ __launch_bounds__(kCopyThreads) void kv_compact_kernel(KvPagesParams p) {
  const int moves = p.plan.head[1], live = p.plan.head[2];
  if (moves == 0) return;
  const int64_t entries = (int64_t)p.rows * p.max_pages;
  const int64_t wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t thread = wg * kCopyThreads + threadIdx.x, threads = (int64_t)gridDim.x * gridDim.y * kCopyThreads;
  for (int64_t i = thread; i < entries; i += threads) {
    const int id = p.table[i];
    if (id >= live && id < p.pool.num_pages) p.table[i] = p.plan.take[id];
  }
  for (int64_t i = thread; i < moves; i += threads) {
    p.refs[p.plan.dst[i]] = p.refs[p.plan.src[i]];
    p.refs[p.plan.src[i]] = 0;
  }
  copy_pages(p.pool, p.plan.src, p.plan.dst, moves);
}

}  // namespace bq

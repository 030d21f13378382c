// Bookkeeping of the cache's pages on the device (sm_103a): growing, forking,
// freeing and compacting rows of a block table, and the copies of pages that
// go with it.
//
// State, all int32 and owned by the caller: ref_counts [NB] (how many table
// entries hold a page; 0 = free), block_tables [S][MB], seq_lens [S] (row s
// holds ceil(seq_lens[s] / bs) pages). There is no free list to keep in
// step: a page is free when its count is 0, and an allocation takes the
// lowest free ids in the order of its requests, so the same state always
// gives the same ids.
//
// The k-th free id is a prefix sum over ref_counts. One thread-block cluster
// does it in one launch: each CTA counts the free pages of its segment, the
// counts meet through distributed shared memory, and each CTA then writes
// its free ids at their ranks. (A pool of 131,072 pages is 512 KiB of counts,
// 64 KiB per CTA of a cluster of 8.) These kernels are bound by latency: a
// launch and a few trips to memory.
#pragma once

#include "pda_kernels.cuh"

namespace pda {

constexpr int kPageThreads = 1024;        // cluster kernels
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageCluster = 8;           // CTAs of the cluster kernels (1 for small pools)
constexpr int kMaxPageArrays = 128;       // cache arrays per launch (kernel parameter space)
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = kCopyThreads * 4 * 16;   // bytes a CTA copies at once

struct PageState {
  int32_t* refs;      // [num_blocks]
  int32_t* tables;    // [num_rows][max_blocks]
  int32_t* lens;      // [num_rows]
  int num_blocks;
  int num_rows;
  int max_blocks;
  int block_size;
};

// Workspace of one page call (ints, see page_ws_layout).
struct PageWs {
  int32_t* head;      // [0]: pages to move (compact)
  int32_t* claims;    // [num_rows]: lowest request that names the row
  int2* reqs;         // [n]: a request's length (-1: refused) and the rank of its first fresh page
  int32_t* fresh;     // [num_blocks]: free ids by rank; compact: target of each moved page
  int32_t* moved;     // [num_blocks]: compact: page to move, by rank
  int32_t* remap;     // [num_blocks]: compact: a page's id after it, -1 for a free page
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Every thread of the cluster meets, and what each wrote (shared or global)
// is seen by all.
__device__ __forceinline__ void cluster_meet() {
  __threadfence();
  cluster_sync();
}

// Exclusive prefix of v over the block's kPageThreads threads; total gets the sum.
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const T before = warp ? warp_sums[warp - 1] : 0;
  total = warp_sums[kPageWarps - 1];
  __syncthreads();
  return before + x - v;
}

// Sum of the cluster's per-CTA counts below this CTA, and of all of them.
// counts: the same shared int in every CTA, written before the last meet.
__device__ __forceinline__ void cluster_prefix(int* count, int& before, int& total) {
  const int me = (int)cluster_rank(), n = (int)cluster_size();
  before = total = 0;
  for (int i = 0; i < n; ++i) {
    const int c = ld_cluster_s32(mapa_cluster(smem_u32(count), i));
    if (i < me) before += c;
    total += c;
  }
}

__device__ __forceinline__ int pages_of(int len, int bs) { return (len + bs - 1) / bs; }

// The ids of [first, end) whose count says free (kFree) or held, in order:
// f(rank, id) for each, ranks counted from `base`. Every thread of the CTA calls it.
template <typename Test, typename F>
__device__ __forceinline__ void each_ranked(int first, int end, int base, int* warp_sums, Test test, F f) {
  for (int i0 = first; i0 < end; i0 += kPageThreads * 4) {
    const int i = i0 + (int)threadIdx.x * 4;
    bool hit[4];
    int n = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      hit[u] = i + u < end && test(i + u);
      n += hit[u] ? 1 : 0;
    }
    int total;
    int r = base + block_prefix(n, warp_sums, total);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (hit[u]) f(r++, i + u);
    base += total;
  }
}

template <typename Test>
__device__ __forceinline__ int count_ids(int first, int end, int* warp_sums, Test test) {
  int n = 0;
  for (int i = first + (int)threadIdx.x; i < end; i += kPageThreads) n += test(i) ? 1 : 0;
  int total;
  (void)block_prefix(n, warp_sums, total);
  return total;
}

// pda_page_alloc_kernel: one cluster serves n requests for fresh pages.
//   grow (children == nullptr): row rows[i] gets add[i] more tokens;
//   fork: row children[i] is to start as a copy of row rows[i], and needs a
//   fresh page when the parent's last page is not full.
// The lowest request that names a row owns it: a later one of the same row
// (or a fork whose parent is a child of the call) is refused. Refused
// requests (also: a row out of range, a child that holds tokens, a length
// past the table row, a page beyond the free ones) set a status bit, change
// nothing and need no page. Request i is short of pages when the needs of
// requests 0..i sum past the free pages.
// Fork leaves the table rows to pda_page_copy_kernel, which has the whole GPU,
// and the children's lengths with them: until the entries and the copied page
// are there, a child's row is empty to whoever reads it in between.
struct AllocParams {
  PageState st;
  PageWs ws;
  const int32_t* rows;
  const int32_t* add;        // grow
  const int32_t* children;   // fork
  int n;
};

__global__ void __launch_bounds__(kPageThreads) pda_page_alloc_kernel(const AllocParams p) {
  __shared__ int warp_sums[kPageWarps];
  __shared__ long long need_sums[kPageWarps];
  __shared__ int count;
  const int me = (int)cluster_rank(), ctas = (int)cluster_size(), tid = threadIdx.x;
  const bool fork = p.children != nullptr;
  const int bs = p.st.block_size, NB = p.st.num_blocks;
  const int seg = (NB + ctas - 1) / ctas;
  const int first = min(NB, me * seg), end = min(NB, first + seg);
  auto is_free = [&](int i) { return __ldcg(p.st.refs + i) == 0; };
  for (int i = me * kPageThreads + tid; i < p.st.num_rows; i += ctas * kPageThreads) p.ws.claims[i] = INT32_MAX;
  const int mine = count_ids(first, end, warp_sums, is_free);
  if (tid == 0) count = mine;
  cluster_meet();
  int base, free_pages;
  cluster_prefix(&count, base, free_pages);

  // Every CTA walks all requests (claims are idempotent), so that each knows
  // how many fresh pages are asked for; CTA 0 writes the records.
  auto in_range = [&](int r) { return (uint32_t)r < (uint32_t)p.st.num_rows; };
  for (int i = tid; i < p.n; i += kPageThreads) {
    const int r = fork ? p.children[i] : p.rows[i];
    if (in_range(r) && p.rows[i] >= 0) atomicMin(p.ws.claims + r, i);
  }
  __threadfence();
  __syncthreads();
  long long need_all = 0;
  for (int i0 = 0; i0 < p.n; i0 += kPageThreads) {
    const int i = i0 + tid;
    int need = 0, len = -1;
    bool padding = false;
    if (i < p.n) {
      const int r = p.rows[i], c = fork ? p.children[i] : r;
      padding = r < 0 || c < 0;
      bool ok = in_range(r) && in_range(c) && __ldcg(p.ws.claims + c) == i;
      if (ok && fork) ok = __ldcg(p.ws.claims + r) == INT32_MAX && __ldcg(p.st.lens + c) == 0;
      if (ok) {
        const int old = __ldcg(p.st.lens + r);
        const long long now = fork ? old : (long long)old + p.add[i];
        ok = old >= 0 && (fork || p.add[i] >= 0) && now <= (long long)p.st.max_blocks * bs;
        if (ok) {
          len = (int)now;
          need = fork ? (old % bs != 0) : pages_of(len, bs) - pages_of(old, bs);
        }
      }
    }
    long long total;
    const long long at = need_all + block_prefix((long long)need, need_sums, total);
    if (need > 0 && at + need > free_pages) len = -1;
    if (i < p.n && me == 0) {
      if (len < 0 && !padding) atomicOr(&g_status, kStatusPageRefused);
      p.ws.reqs[i] = make_int2(len, (int)min(at, (long long)free_pages));
    }
    need_all += total;
  }
  const int wanted = (int)min(need_all, (long long)free_pages);
  if (base < wanted)
    each_ranked(first, end, base, warp_sums, is_free, [&](int r, int id) {
      if (r < wanted) p.ws.fresh[r] = id;
    });
  cluster_meet();
  grid_dependents_launch();

  // apply: a warp per request
  const int lane = tid & 31;
  for (int i = me * kPageWarps + (tid >> 5); i < p.n; i += ctas * kPageWarps) {
    const int2 q = __ldcg(p.ws.reqs + i);
    if (q.x < 0) continue;
    const int r = fork ? p.children[i] : p.rows[i];
    if (fork) {
      if (q.x % bs != 0 && lane == 0) p.st.refs[__ldcg(p.ws.fresh + q.y)] = 1;
    } else {
      const int from = pages_of(__ldcg(p.st.lens + r), bs), to = pages_of(q.x, bs);
      for (int j = from + lane; j < to; j += 32) {
        const int id = __ldcg(p.ws.fresh + q.y + (j - from));
        p.st.tables[(size_t)r * p.st.max_blocks + j] = id;
        p.st.refs[id] = 1;
      }
      __syncwarp();
    }
    if (lane == 0 && !fork) p.st.lens[r] = q.x;
  }
}

// Copies of whole pages in up to kMaxPageArrays arrays, kCopyChunk bytes per
// CTA at a time with four 16-byte loads in flight per thread, over the whole
// GPU; the first CTAs do the fork's or the compaction's table entries.
// Bound: bytes.
struct PageArray {
  uint8_t* base;
  long long bytes;     // of one page, a multiple of 16
};
enum : int { kCopyPairs = 0, kCopyFork = 1, kCopyCompact = 2 };
struct CopyParams {
  PageState st;
  PageWs ws;
  const int32_t* src;        // kCopyPairs
  const int32_t* dst;
  const int32_t* rows;       // kCopyFork: parents
  const int32_t* children;
  int n;                     // pairs or forks (compact: the count is ws.head[0])
  int mode;
  int tables;                // this launch does the table entries too
  int num_arrays;
  int chunks;                // chunks of the largest page
  PageArray arrays[kMaxPageArrays];
};

__device__ __forceinline__ bool page_pair(const CopyParams& p, int i, int& src, int& dst) {
  if (p.mode == kCopyPairs) {
    src = __ldg(p.src + i);
    dst = __ldg(p.dst + i);
    if (src < 0 || dst < 0 || src == dst) return false;
  } else if (p.mode == kCopyFork) {
    const int2 q = __ldcg(p.ws.reqs + i);
    if (q.x < 0 || q.x % p.st.block_size == 0) return false;
    src = __ldcg(p.st.tables + (size_t)__ldg(p.rows + i) * p.st.max_blocks + q.x / p.st.block_size);
    dst = __ldcg(p.ws.fresh + q.y);
  } else {
    src = __ldcg(p.ws.moved + i);
    dst = __ldcg(p.ws.fresh + i);
  }
  if ((uint32_t)src >= (uint32_t)p.st.num_blocks || (uint32_t)dst >= (uint32_t)p.st.num_blocks) {
    atomicOr(&g_status, kStatusBadBlock);
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kCopyThreads) pda_page_copy_kernel(const __grid_constant__ CopyParams p) {
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int bs = p.st.block_size, MB = p.st.max_blocks;
  if (p.tables && p.mode == kCopyFork) {
    // a warp takes 128 entries of one fork's row at a time
    const int parts = (MB + 127) / 128;
    const long long items = (long long)p.n * parts;
    for (long long it = (long long)blockIdx.x * (kCopyThreads / 32) + (tid >> 5); it < items;
         it += (long long)gridDim.x * (kCopyThreads / 32)) {
      const int i = (int)(it / parts), j0 = (int)(it % parts) * 128;
      const int2 q = __ldcg(p.ws.reqs + i);
      if (q.x < 0) continue;
      const int full = q.x / bs, np = pages_of(q.x, bs);
      if (j0 == 0 && (tid & 31) == 0) p.st.lens[__ldg(p.children + i)] = q.x;
      const int32_t* from = p.st.tables + (size_t)__ldg(p.rows + i) * MB;
      int32_t* to = p.st.tables + (size_t)__ldg(p.children + i) * MB;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + 32 * u + (tid & 31);
        if (j >= np) continue;
        int id;
        if (j < full) {
          id = __ldcg(from + j);
          if ((uint32_t)id < (uint32_t)p.st.num_blocks)
            atomicAdd(p.st.refs + id, 1);
          else
            atomicOr(&g_status, kStatusBadBlock);
        } else {
          id = __ldcg(p.ws.fresh + q.y);
        }
        to[j] = id;
      }
    }
  } else if (p.tables && p.mode == kCopyCompact) {
    const long long items = (long long)p.st.num_rows * MB;
    for (long long it = (long long)blockIdx.x * kCopyThreads + tid; it < items; it += (long long)gridDim.x * kCopyThreads) {
      const int s = (int)(it / MB), j = (int)(it % MB);
      if (j >= pages_of(__ldg(p.st.lens + s), bs)) continue;
      const int id = p.st.tables[it];
      if ((uint32_t)id >= (uint32_t)p.st.num_blocks) {
        atomicOr(&g_status, kStatusBadBlock);
        continue;
      }
      const int to = __ldcg(p.ws.remap + id);
      if (to < 0)
        atomicOr(&g_status, kStatusPageRefused);   // the entry names a free page
      else if (to != id)
        p.st.tables[it] = to;
    }
  }
  const int n = p.mode == kCopyCompact ? __ldcg(p.ws.head) : p.n;
  const long long items = (long long)n * p.num_arrays * p.chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int c = (int)(it % p.chunks);
    const long long rest = it / p.chunks;
    const int a = (int)(rest % p.num_arrays);
    int src, dst;
    if (!page_pair(p, (int)(rest / p.num_arrays), src, dst)) continue;
    const long long bytes = p.arrays[a].bytes;
    const uint4* from = reinterpret_cast<const uint4*>(p.arrays[a].base + src * bytes + (long long)c * kCopyChunk);
    uint4* to = reinterpret_cast<uint4*>(p.arrays[a].base + dst * bytes + (long long)c * kCopyChunk);
    const long long left = (bytes - (long long)c * kCopyChunk) / 16;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u * kCopyThreads + tid < left) v[u] = __ldcs(from + u * kCopyThreads + tid);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u * kCopyThreads + tid < left) __stcs(to + u * kCopyThreads + tid, v[u]);
  }
}

// pda_page_free_kernel: one CTA per row. The length is taken with an
// exchange, so a row named twice is freed once.
struct FreeParams {
  PageState st;
  const int32_t* rows;
  int n;
};
__global__ void __launch_bounds__(128) pda_page_free_kernel(const FreeParams p) {
  __shared__ int len;
  const int r = __ldg(p.rows + blockIdx.x);
  if (r < 0) return;   // padding
  if ((uint32_t)r >= (uint32_t)p.st.num_rows) {
    if (threadIdx.x == 0) atomicOr(&g_status, kStatusPageRefused);
    return;
  }
  if (threadIdx.x == 0) len = atomicExch(p.st.lens + r, 0);
  __syncthreads();
  const int np = len > 0 ? min(pages_of(len, p.st.block_size), p.st.max_blocks) : 0;
  for (int j = threadIdx.x; j < np; j += 128) {
    const int id = p.st.tables[(size_t)r * p.st.max_blocks + j];
    if ((uint32_t)id >= (uint32_t)p.st.num_blocks) {
      atomicOr(&g_status, kStatusBadBlock);
    } else if (atomicSub(p.st.refs + id, 1) <= 0) {
      atomicAdd(p.st.refs + id, 1);            // the page was free already
      atomicOr(&g_status, kStatusPageRefused);
    }
  }
}

// pda_page_compact_kernel: with L live pages, the k-th free id below L takes
// the k-th live page at or above L; the two are equally many. Writes the
// moves (pda_page_copy_kernel makes them), every page's id after them (-1 for a
// free page, which no table entry in use may name) and the counts' new places.
struct CompactParams {
  PageState st;
  PageWs ws;
  int32_t* new_ids;    // [num_blocks], or nullptr
};
__global__ void __launch_bounds__(kPageThreads) pda_page_compact_kernel(const CompactParams p) {
  __shared__ int warp_sums[kPageWarps];
  __shared__ int count, holes, movers;
  const int me = (int)cluster_rank(), ctas = (int)cluster_size(), tid = threadIdx.x;
  const int NB = p.st.num_blocks;
  const int seg = (NB + ctas - 1) / ctas;
  const int first = min(NB, me * seg), end = min(NB, first + seg);
  auto held = [&](int i) { return __ldcg(p.st.refs + i) > 0; };
  const int mine = count_ids(first, end, warp_sums, held);
  if (tid == 0) count = mine;
  cluster_meet();
  int before, live;
  cluster_prefix(&count, before, live);
  auto is_hole = [&](int i) { return i < live && !held(i); };
  auto is_mover = [&](int i) { return i >= live && held(i); };
  const int nh = count_ids(first, end, warp_sums, is_hole);
  const int nm = count_ids(first, end, warp_sums, is_mover);
  if (tid == 0) {
    holes = nh;
    movers = nm;
  }
  cluster_meet();
  int hole0, mover0, all;
  cluster_prefix(&holes, hole0, all);
  cluster_prefix(&movers, mover0, all);
  if (nh) each_ranked(first, end, hole0, warp_sums, is_hole, [&](int r, int id) { p.ws.fresh[r] = id; });
  if (nm) each_ranked(first, end, mover0, warp_sums, is_mover, [&](int r, int id) { p.ws.moved[r] = id; });
  for (int i = first + tid; i < end; i += kPageThreads) {
    if (is_mover(i)) continue;
    p.ws.remap[i] = held(i) ? i : -1;
    if (p.new_ids) p.new_ids[i] = i;
  }
  if (me == 0 && tid == 0) {
    p.ws.head[0] = all;
  }
  cluster_meet();
  grid_dependents_launch();
  for (int k = me * kPageThreads + tid; k < all; k += ctas * kPageThreads) {
    const int id = __ldcg(p.ws.moved + k), to = __ldcg(p.ws.fresh + k);
    p.ws.remap[id] = to;
    if (p.new_ids) p.new_ids[id] = to;
    p.st.refs[to] = __ldcg(p.st.refs + id);
    p.st.refs[id] = 0;
  }
}

}  // namespace pda

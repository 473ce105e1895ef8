// kvq_pages.cu -- a pool of pages kept on the device (references, a stack of
// free pages), sequences that fork, grow and go, and the rows of an accepted
// path of drafted tokens moved together.
//
// These kernels move little (a fork copies the rows of one partly filled page, a
// commit a few rows) and are bound by latency: a launch and a chain of dependent
// loads.  So each is one launch, and what has to be in order across a launch is
// found by counting, not by waiting: a child's or an entry's place in the order is
// the number of those before it, which every block counts for itself; the block
// that finishes last (a counter in the pool's state) changes what the others have
// read.  No result depends on the order of atomics.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPgThreads = 256;
constexpr int kPgScanThreads = 1024;

__device__ __forceinline__ void flag(int32_t *err_flags, int32_t bit) {
  if (err_flags) atomicOr(err_flags, bit);
}

// Whether this block is the last of the grid to get here (all threads of the
// block; the counter is 0 again afterwards).  What the blocks read and wrote
// before is finished for the last one.  The counter's upper bits add up the
// blocks' `mine` (thread 0's), its lower kBits count them; `all` gets the sum.
template <int kBits>
__device__ bool last_block(int32_t *counter, uint32_t mine, uint32_t *all) {
  __shared__ uint32_t last, sum;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t now =
        atomicAdd(reinterpret_cast<uint32_t *>(counter), 1u + (mine << kBits)) + 1u + (mine << kBits);
    last = (now & ((1u << kBits) - 1u)) == gridDim.x;
    sum = now >> kBits;
    if (last) *counter = 0;
    __threadfence();
  }
  __syncthreads();
  *all = sum;
  return last != 0u;
}

// Inclusive sums over a warp.
__device__ __forceinline__ int warp_scan(int n) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, n, off);
    if (lane >= off) n += v;
  }
  return n;
}

// Sum over the threads before this one; `total` gets the sum over the block.
template <int kThreads>
__device__ __forceinline__ int block_before(int n, int *total) {
  __shared__ int warps[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inc = warp_scan(n);
  __syncthreads();                                      // (the last round's sums have been read)
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  int before = inc - n, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = warps[w];
    if (w < warp) before += v;
    all += v;
  }
  *total = all;
  return before;
}

// ---------------------------------------------------------------------------
// Pages from the pool.  One block: 1,024 requests at a time, their counts summed,
// then a thread per page.
__global__ void __launch_bounds__(kPgScanThreads)
pages_alloc_kernel(const kvq_page_pool pool, int32_t *tables, int32_t n, int32_t width,
                   const int32_t *begin, const int32_t *end, int32_t *err_flags) {
  __shared__ int first[kPgScanThreads], at[kPgScanThreads], given_end;
  const int tid = threadIdx.x;
  allow_dependents_launch();
  grid_dependency_wait();
  const int num_free = min(max(pool.state[0], 0), pool.num_pages);
  int64_t before = 0;                                   // wanted by the requests before
  int taken = 0;
  bool out = false;                                     // a request has not fitted
  for (int r0 = 0; r0 < n; r0 += kPgScanThreads) {
    const int r = r0 + tid;
    int b = 0, need = 0;
    if (r < n) {
      b = begin[r];
      const int e = end[r];
      if (b < 0 || e < b || e > width) flag(err_flags, KVQ_ERRF_CONTEXT_RANGE);
      else need = e - b;
    }
    // (a sum over 1,024 tables of fewer than 2^21 entries each stays in 31 bits)
    int total;
    const int mine = block_before<kPgScanThreads>(need, &total);
    if (tid == 0) given_end = num_free;
    first[tid] = mine;
    at[tid] = b;
    __syncthreads();
    // the first request that does not fit, and all that want pages after it, get none
    if (need > 0 && before + mine + need > num_free) {
      atomicMin(&given_end, static_cast<int>(min(before + mine, static_cast<int64_t>(num_free))));
      flag(err_flags, KVQ_ERRF_NO_PAGES);
    }
    __syncthreads();
    const int64_t stop = given_end;
    for (int k = tid; k < total; k += kPgScanThreads) {
      int lo = 0, hi = kPgScanThreads - 1;              // the last request that starts at k or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      int page = -1;
      if (before + k < stop) {
        page = pool.free_pages[num_free - 1 - (before + k)];
        if (page >= 0 && page < pool.num_pages) pool.ref_counts[page] = 1;
      }
      tables[static_cast<int64_t>(r0 + lo) * width + at[lo] + (k - first[lo])] = page;
    }
    before += total;
    if (!out) taken = static_cast<int>(min(before, stop));
    out = out || before > stop;
    __syncthreads();
  }
  if (tid == 0) pool.state[0] = num_free - taken;
}

// ---------------------------------------------------------------------------
// References given back, a block per request; the last block collects the pages
// that reached 0, which the others have marked, in ascending order.
constexpr int kPgFreeThreads = 512;

__global__ void __launch_bounds__(kPgFreeThreads)
pages_free_kernel(const kvq_page_pool pool, const int32_t *tables, int32_t width,
                  const int32_t *begin, const int32_t *end, int32_t *err_flags) {
  const int tid = threadIdx.x;
  allow_dependents_launch();
  grid_dependency_wait();
  const int64_t r = blockIdx.x;
  const int b = begin[r], e = end[r];
  if (b < 0 || e < b || e > width) {
    if (tid == 0) flag(err_flags, KVQ_ERRF_CONTEXT_RANGE);
  } else {
    for (int i = b + tid; i < e; i += kPgFreeThreads) {
      const int page = tables[r * width + i];
      if (page < 0) continue;
      if (page >= pool.num_pages) {
        flag(err_flags, KVQ_ERRF_BLOCK_RANGE);
        continue;
      }
      const int held = atomicSub(pool.ref_counts + page, 1);
      if (held == 1) {
        atomicOr(pool.marks + (page >> 5), 1 << (page & 31));
      } else if (held < 1) {
        atomicAdd(pool.ref_counts + page, 1);
        flag(err_flags, KVQ_ERRF_PAGE_STATE);
      }
    }
  }
  uint32_t none;
  if (!last_block<31>(pool.state + 1, 0u, &none)) return;
  const int words = (pool.num_pages + 31) / 32;
  int num_free = min(max(pool.state[0], 0), pool.num_pages);
  uint32_t next = tid < words ? static_cast<uint32_t>(__ldcg(pool.marks + tid)) : 0u;
  for (int w0 = 0; w0 < words; w0 += kPgFreeThreads) {
    uint32_t mark = next;
    const int w = w0 + tid;
    next = w + kPgFreeThreads < words
               ? static_cast<uint32_t>(__ldcg(pool.marks + w + kPgFreeThreads)) : 0u;
    if (__syncthreads_or(mark != 0u) == 0) continue;
    int total;
    int to = num_free + block_before<kPgFreeThreads>(__popc(mark), &total);
    if (mark != 0u) pool.marks[w] = 0;
    while (mark != 0u) {
      const int bit = __ffs(mark) - 1;
      mark &= mark - 1;
      if (to < pool.num_pages) pool.free_pages[to] = 32 * w + bit;
      ++to;
    }
    num_free = min(num_free + total, pool.num_pages);
  }
  if (tid == 0) pool.state[0] = num_free;
}

// ---------------------------------------------------------------------------
// Forks: `splits` blocks a child, which share the copy of its last page; the first
// of them writes the child's table.
struct ForkParams {
  kvq_cache c;
  kvq_page_pool pool;
  const int32_t *parents, *tables, *lens;
  int32_t *child_tables, *child_lens, *err_flags;
  int32_t children, num_parents, width, log2_bs, splits;
};

// Child i's parent, or -1, and its length.
__device__ __forceinline__ int fork_parent(const ForkParams &p, int i, int *len) {
  const int parent = p.parents[i];
  *len = 0;
  if (parent < 0 || parent >= p.num_parents) return -1;
  const int L = p.lens[parent];
  if (L < 0 || L > (static_cast<int64_t>(p.width) << p.log2_bs)) return -1;
  *len = L;
  return parent;
}

template <typename T>
__device__ __forceinline__ void copy_part(T *dst, const T *src, int64_t n, int part, int parts) {
  constexpr int kBatch = 4;
  const int64_t step = static_cast<int64_t>(kPgThreads) * parts;
  for (int64_t i = static_cast<int64_t>(part) * kPgThreads + threadIdx.x; i < n; i += kBatch * step) {
    T v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k * step < n) v[k] = src[i + k * step];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k * step < n) dst[i + k * step] = v[k];
  }
}

__global__ void __launch_bounds__(kPgThreads) pages_fork_kernel(const ForkParams p) {
  const int tid = threadIdx.x;
  const int i = static_cast<int>(blockIdx.x) / p.splits;
  const int part = static_cast<int>(blockIdx.x) - i * p.splits;
  const int bs = 1 << p.log2_bs;
  allow_dependents_launch();
  grid_dependency_wait();
  const int num_free = min(max(p.pool.state[0], 0), p.pool.num_pages);
  // Children before this one that take a page: for their parents' last ones, partly filled
  // and the pool's.
  auto held = [&](int page) -> bool { return page >= 0 && page < p.pool.num_pages; };
  int rank = 0;
  for (int j0 = 0; j0 < i; j0 += kPgThreads) {
    const int j = j0 + tid;
    bool takes = false;
    if (j < i) {
      int l;
      const int of = fork_parent(p, j, &l);
      if ((l & (bs - 1)) != 0)
        takes = held(p.tables[static_cast<int64_t>(of) * p.width + (l >> p.log2_bs)]);
    }
    rank += __syncthreads_count(takes);
  }
  int len;
  int parent = fork_parent(p, i, &len);
  if (parent < 0 && part == 0 && tid == 0) {
    const int want = p.parents[i];
    if (want >= p.num_parents) flag(p.err_flags, KVQ_ERRF_PATH_RANGE);
    else if (want >= 0) flag(p.err_flags, KVQ_ERRF_CONTEXT_RANGE);
  }
  const int rest = len & (bs - 1), full = len >> p.log2_bs;
  if (rest != 0 && rank >= num_free && held(p.tables[static_cast<int64_t>(parent) * p.width + full])) {
    if (part == 0 && tid == 0) flag(p.err_flags, KVQ_ERRF_NO_PAGES);
    parent = -1;
  }
  bool takes = false;
  if (part == 0 && tid == 0) p.child_lens[i] = parent < 0 ? 0 : len;
  if (parent >= 0) {
    const int32_t *from = p.tables + static_cast<int64_t>(parent) * p.width;
    int32_t *to = p.child_tables + static_cast<int64_t>(i) * p.width;
    if (part == 0) {
      for (int k = tid; k < full; k += kPgThreads) {
        const int page = from[k];
        to[k] = page;
        if (held(page)) atomicAdd(p.pool.ref_counts + page, 1);
        else flag(p.err_flags, KVQ_ERRF_BLOCK_RANGE);
      }
    }
    if (rest != 0) {
      // (a parent's page outside the pool is passed on.  Read here, not with the parent's
      // length: with the read up there a fork 1 -> 8 took 2 us more)
      const int src = from[full];
      takes = held(src);
      const int dst = takes ? p.pool.free_pages[num_free - 1 - rank] : src;
      const bool ok = takes && held(dst);
      if (part == 0 && tid == 0) {
        to[full] = dst;
        if (ok) p.pool.ref_counts[dst] = 1;
        else flag(p.err_flags, KVQ_ERRF_BLOCK_RANGE);
      }
      if (ok) {
        // a page's rows lie one behind the other
        const int64_t a = static_cast<int64_t>(src) << p.log2_bs, b = static_cast<int64_t>(dst) << p.log2_bs;
        const int64_t H = p.c.num_kv_heads, row16 = H * (kHeadDim / 16);
        uint4 *kc = reinterpret_cast<uint4 *>(p.c.k_codes), *vc = reinterpret_cast<uint4 *>(p.c.v_codes);
        copy_part(kc + b * row16, kc + a * row16, rest * row16, part, p.splits);
        copy_part(vc + b * row16, vc + a * row16, rest * row16, part, p.splits);
        copy_part(p.c.k_scales + b * H, p.c.k_scales + a * H, rest * H, part, p.splits);
        copy_part(p.c.v_scales + b * H, p.c.v_scales + a * H, rest * H, part, p.splits);
      }
    }
  }
  // (at most 2^12 children, 2^12 blocks or a few an SM)
  uint32_t taken;
  if (!last_block<16>(p.pool.state + 1, takes && part == 0 ? 1u : 0u, &taken)) return;
  if (tid == 0) p.pool.state[0] = num_free - static_cast<int>(taken);
}

// ---------------------------------------------------------------------------
// The rows of an accepted path moved together, a block per request.  A thread owns
// 16 bytes of a row (or a scale) and moves them for all nodes in ascending order:
// the place of node a, base + a, is never behind the place that a later node is
// read from, base + path[a'] >= base + a' > base + a, so nothing is overwritten
// before it is read and the threads need not wait for one another.
constexpr int kPgCommitThreads = 256;

struct CommitParams {
  kvq_cache c;
  const int32_t *paths, *counts, *tables, *lens;
  int32_t *new_lens, *err_flags;
  int32_t R, width, log2_bs;
  int64_t num_blocks;
};

template <typename T>
__device__ __forceinline__ void commit_rows(T *plane, int64_t pitch, int at, const int64_t *src,
                                            const int64_t *dst, int n) {
  constexpr int kBatch = 8;
  for (int a0 = 0; a0 < n; a0 += kBatch) {
    T v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (a0 + k < n) v[k] = plane[src[a0 + k] * pitch + at];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (a0 + k < n) plane[dst[a0 + k] * pitch + at] = v[k];
  }
}

__global__ void __launch_bounds__(kPgCommitThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int64_t src[kTreeMaxNodes], dst[kTreeMaxNodes];
  __shared__ int kept;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  allow_dependents_launch();
  grid_dependency_wait();
  const int L = p.lens[r], count = p.counts[r];
  const int64_t cap = static_cast<int64_t>(p.width) << p.log2_bs;
  const bool idle = L == 0 && count == 0;
  const bool in_range = idle || (L >= p.R && L <= cap);
  bool path_ok = count >= 0 && count <= p.R;
  const int n = path_ok && in_range ? count : 0;
  const int32_t *path = p.paths + r * p.R;
  const int32_t *table = p.tables + r * p.width;
  const int base = L - p.R;
  const int shift = p.log2_bs, low = (1 << p.log2_bs) - 1;
  bool bad_page = false;
  for (int a = tid; a < n; a += kPgCommitThreads) {
    const int node = path[a];
    const bool ok = node >= 0 && node < p.R && (a == 0 || path[a - 1] < node);
    path_ok = path_ok && ok;
    // (a node that stays where it is keeps its row: source and place are the same)
    const int from = base + (ok ? node : a), to = base + a;
    const int64_t fp = table[from >> shift], tp = table[to >> shift];
    if (fp < 0 || fp >= p.num_blocks || tp < 0 || tp >= p.num_blocks) bad_page = true;
    src[a] = (fp << shift) + (from & low);
    dst[a] = (tp << shift) + (to & low);
  }
  const bool paths_bad = __syncthreads_or(!path_ok) != 0;
  const bool pages_bad = __syncthreads_or(bad_page) != 0;
  if (tid == 0) {
    p.new_lens[r] = idle ? 0 : (paths_bad || !in_range ? L : base + count);
    if (!in_range) flag(p.err_flags, KVQ_ERRF_CONTEXT_RANGE);
    else if (paths_bad) flag(p.err_flags, KVQ_ERRF_PATH_RANGE);
    if (pages_bad && !paths_bad) flag(p.err_flags, KVQ_ERRF_BLOCK_RANGE);
  }
  if (paths_bad || n == 0) return;
  int m = n;
  if (pages_bad) {
    // rows of pages outside the cache leave the list (rare)
    if (tid == 0) {
      const int64_t slots = p.num_blocks << shift;
      int k = 0;
      for (int a = 0; a < n; ++a)
        if (src[a] >= 0 && src[a] < slots && dst[a] >= 0 && dst[a] < slots) {
          src[k] = src[a];
          dst[k++] = dst[a];
        }
      kept = k;
    }
    __syncthreads();
    m = kept;
  }
  const int H = p.c.num_kv_heads, row16 = H * (kHeadDim / 16);
  uint4 *kc = reinterpret_cast<uint4 *>(p.c.k_codes), *vc = reinterpret_cast<uint4 *>(p.c.v_codes);
  for (int at = tid; at < 2 * row16 + 2 * H; at += kPgCommitThreads) {
    if (at < row16) commit_rows(kc, row16, at, src, dst, m);
    else if (at < 2 * row16) commit_rows(vc, row16, at - row16, src, dst, m);
    else if (at < 2 * row16 + H) commit_rows(p.c.k_scales, H, at - 2 * row16, src, dst, m);
    else commit_rows(p.c.v_scales, H, at - 2 * row16 - H, src, dst, m);
  }
}

}  // namespace

cudaError_t launch_pages_alloc(const kvq_page_pool &pool, int32_t *tables, int32_t n, int32_t width,
                               const int32_t *begin, const int32_t *end, int32_t *err_flags,
                               cudaStream_t stream) {
  return launch_overlapped(pages_alloc_kernel, dim3(1), dim3(kPgScanThreads), 0, stream, pool,
                           tables, n, width, begin, end, err_flags);
}

cudaError_t launch_pages_free(const kvq_page_pool &pool, const int32_t *tables, int32_t n,
                              int32_t width, const int32_t *begin, const int32_t *end,
                              int32_t *err_flags, cudaStream_t stream) {
  return launch_overlapped(pages_free_kernel, dim3(static_cast<unsigned>(n)), dim3(kPgFreeThreads),
                           0, stream, pool, tables, width, begin, end, err_flags);
}

cudaError_t launch_pages_fork(const kvq_cache &c, const kvq_page_pool &pool, const int32_t *parents,
                              int32_t children, const int32_t *tables, int32_t num_parents,
                              int32_t width, const int32_t *lens, int32_t log2_block,
                              int32_t *child_tables, int32_t *child_lens, int32_t *err_flags,
                              int32_t sms, cudaStream_t stream) {
  ForkParams p{c, pool, parents, tables, lens, child_tables, child_lens, err_flags, children,
               num_parents, width, log2_block, 1};
  // blocks a child: a page of 16-byte pieces over 256 threads, 4 at a time, as far as
  // there are SMs for it
  const int64_t pieces = (static_cast<int64_t>(c.num_kv_heads) * (kHeadDim / 16)) << log2_block;
  const int64_t useful = (pieces + 4 * kPgThreads - 1) / (4 * kPgThreads);
  p.splits = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(useful, 4LL * sms / children)));
  return launch_overlapped(pages_fork_kernel, dim3(static_cast<unsigned>(children * p.splits)),
                           dim3(kPgThreads), 0, stream, p);
}

cudaError_t launch_tree_commit(const kvq_cache &c, const int32_t *paths, const int32_t *counts,
                               int32_t n, int32_t R, const int32_t *tables, int32_t width,
                               int32_t log2_block, const int32_t *lens, int32_t *new_lens,
                               int32_t *err_flags, cudaStream_t stream) {
  const CommitParams p{c, paths, counts, tables, lens, new_lens, err_flags, R, width, log2_block,
                       c.num_slots >> log2_block};
  return launch_overlapped(tree_commit_kernel, dim3(static_cast<unsigned>(n)),
                           dim3(kPgCommitThreads), 0, stream, p);
}

}  // namespace kvq

// Forking, freeing and compacting the pages of a paged cache (sm_100a).
//
// A page is in use when an entry among the first ceil(len / page_size) of some sequence's row of
// the block table names it.  Everything here follows from the block table and the lengths, so no
// reference counts are kept between calls:
//   fork:    new sequence i continues sequence parent[i].  Pages that are full are shared; a last
//            page that is not full stays with the first new sequence that ends in it, and every
//            other one gets a copy in a free page (also the first, if the page is full in some
//            other row).  Pages that no new row names are free.
//   compact: the k-th page in use at or after the number of pages in use moves to the k-th free
//            page before it.
// Free pages are handed out in ascending order and copies in the order of the new sequences, so
// results do not depend on the order of the atomics (a minimum per page).
//
// Bound by HBM where pages are copied (2 bytes moved a byte), and by latency where only tables
// change: one kernel plans (five of them, one with a single CTA, took FORK1 us on 16 prompts forked
// into 64 sequences, this one and the copies FORK2 us), one copies.
#pragma once

#include "fa_device.cuh"

namespace fa {

constexpr int kMaxPools = 128;
constexpr int kFreeMark = 0x7FFFFFFF;

struct PoolList {
  uint8_t* base[kMaxPools];
  unsigned bytes[kMaxPools];  // of one page
  int n;
};

struct ForkParams {
  const int32_t *table, *lens, *parent;
  int32_t *table_out, *lens_out, *free_pages, *n_free;
  int32_t *mark;          // [num_pages]
  int32_t *rank;          // [R]: number of the copy that row i needs, or -1
  int32_t *src, *dst;     // [R]: the copies
  int32_t *count;         // number of copies
  int32_t *counts;        // per CTA of the planning cluster
  int B, R, max_pages, page_shift, num_pages;
};

struct CompactParams {
  const int32_t *table, *lens;
  int32_t *table_out, *n_live;
  int32_t *mark;       // [num_pages]
  int32_t *src, *dst;  // [num_pages / 2 + 1]
  int32_t *count, *counts;
  int B, max_pages, page_shift, num_pages;
};

// Length of a sequence, or 0 (recorded) for one that the table cannot hold.
__device__ __forceinline__ int pages_len(const int32_t* lens, int b, int max_pages, int page_shift) {
  const int n = __ldg(lens + b);
  if (n < 0 || (long long)n > (long long)max_pages << page_shift) {
    atomicOr(&g_error_word, kErrBadSeqlens);
    return 0;
  }
  return n;
}

__device__ __forceinline__ int fork_len(const ForkParams& p, int i, int* parent) {
  const int b = __ldg(p.parent + i);
  *parent = b;
  if (b < -1 || b >= p.B) {
    atomicOr(&g_error_word, kErrBadSeqlens);
    *parent = -1;
  }
  return *parent < 0 ? 0 : pages_len(p.lens, b, p.max_pages, p.page_shift);
}

__device__ __forceinline__ bool pages_ok(int page, int num_pages) {
  if (page >= 0 && page < num_pages) return true;
  atomicOr(&g_error_word, kErrBadPage);
  return false;
}

// The planning kernels run as one cluster of 8 CTAs, whose barriers (hardware ones) separate their
// steps; pages and rows are cut into 8 contiguous segments, so that ranks are sums over segments.
constexpr int kPlanCtas = 8, kPlanThreads = 1024;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int plan_begin(int n, int cta) { return (int)((long long)n * cta / kPlanCtas); }

// Exclusive rank of one flag per thread over the CTA; the CTA's total in *total.
__device__ __forceinline__ int block_rank(bool flag, int* sm, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned ballot = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sm[warp] = __popc(ballot);
  __syncthreads();
  const int c = sm[lane];
  *total = __reduce_add_sync(0xffffffffu, c);
  return __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + __popc(ballot & ((1u << lane) - 1u));
}

// Per-CTA counts in the workspace: what comes before this CTA, and the total.
__device__ __forceinline__ int plan_before(const int32_t* counts, int cta, int* total) {
  int before = 0, all = 0;
  for (int c = 0; c < kPlanCtas; ++c) {
    const int x = __ldcg(counts + c);
    before += c < cta ? x : 0;
    all += x;
  }
  *total = all;
  return before;
}

// The page of row i's last tokens if that page is not full, else -1.
__device__ __forceinline__ int fork_tail(const ForkParams& p, int i) {
  int b;
  const int n = fork_len(p, i, &b);
  if ((n & ((1 << p.page_shift) - 1)) == 0) return -1;
  return __ldg(p.table + (long long)b * p.max_pages + (n >> p.page_shift));
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  __shared__ int sm[32];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = cta * kPlanThreads + threadIdx.x, threads = kPlanCtas * kPlanThreads;
  const int psm = (1 << p.page_shift) - 1;
  for (int g = tid; g < p.num_pages; g += threads) p.mark[g] = kFreeMark;
  cluster_sync();
  // mark[page]: -1 where some new row holds it full, else the first new row that ends in it
  for (int i = cta * 32 + warp; i < p.R; i += kPlanCtas * 32) {
    int b;
    const int n = fork_len(p, i, &b), full = n >> p.page_shift, np = full + ((n & psm) != 0);
    for (int t = lane; t < np; t += 32) {
      const int page = __ldg(p.table + (long long)b * p.max_pages + t);
      if (pages_ok(page, p.num_pages)) atomicMin(p.mark + page, t < full ? -1 : i);
    }
  }
  cluster_sync();
  // count the copies that this CTA's rows need and the free pages in its part of the pool
  auto needs_copy = [&](int i, int page) { return page >= 0 && page < p.num_pages && __ldcg(p.mark + page) != i; };
  const int i0 = plan_begin(p.R, cta), i1 = plan_begin(p.R, cta + 1);
  const int g0 = plan_begin(p.num_pages, cta), g1 = plan_begin(p.num_pages, cta + 1);
  int copies = 0, frees = 0, total;
  for (int at = i0; at < i1; at += kPlanThreads) {
    const int i = at + threadIdx.x;
    block_rank(i < i1 && needs_copy(i, fork_tail(p, i)), sm, &total);
    copies += total;
  }
  for (int at = g0; at < g1; at += kPlanThreads) {
    const int g = at + threadIdx.x;
    block_rank(g < g1 && __ldcg(p.mark + g) == kFreeMark, sm, &total);
    frees += total;
  }
  if (threadIdx.x == 0) {
    p.counts[cta] = copies;
    p.counts[kPlanCtas + cta] = frees;
  }
  cluster_sync();
  int need, have;
  int r = plan_before(p.counts, cta, &need), f = plan_before(p.counts + kPlanCtas, cta, &have);
  for (int at = i0; at < i1; at += kPlanThreads) {
    const int i = at + threadIdx.x, page = i < i1 ? fork_tail(p, i) : -1;
    const bool copy = i < i1 && needs_copy(i, page);
    const int mine = r + block_rank(copy, sm, &total);
    if (i < i1) p.rank[i] = copy ? mine : -1;
    if (copy) p.src[mine] = page;
    r += total;
  }
  for (int at = g0; at < g1; at += kPlanThreads) {
    const int g = at + threadIdx.x;
    const bool is_free = g < g1 && __ldcg(p.mark + g) == kFreeMark;
    const int mine = f + block_rank(is_free, sm, &total);
    if (is_free) {
      if (mine < need) p.dst[mine] = g;
      else p.free_pages[mine - need] = g;
    }
    f += total;
  }
  const int left = max(have - need, 0);
  for (int k = left + tid; k < p.num_pages; k += threads) p.free_pages[k] = -1;
  if (tid == 0) {
    *p.n_free = left;
    *p.count = min(need, have);
    if (need > have) atomicOr(&g_error_word, kErrNoPages);
  }
  cluster_sync();
  for (int i = cta * 32 + warp; i < p.R; i += kPlanCtas * 32) {
    const int k = __ldcg(p.rank + i);
    int b;
    int n = fork_len(p, i, &b);
    if (k >= have) n = 0;  // no page was left for it
    const int full = n >> p.page_shift, np = full + ((n & psm) != 0);
    const int32_t* from = p.table + (long long)max(b, 0) * p.max_pages;
    int32_t* to = p.table_out + (long long)i * p.max_pages;
    for (int t = lane; t < p.max_pages; t += 32)
      to[t] = t >= np ? -1 : t == full && k >= 0 ? __ldcg(p.dst + k) : __ldg(from + t);
    if (lane == 0) p.lens_out[i] = n;
  }
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  __shared__ int sm[32];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = cta * kPlanThreads + threadIdx.x, threads = kPlanCtas * kPlanThreads;
  const int psm = (1 << p.page_shift) - 1;
  for (int g = tid; g < p.num_pages; g += threads) p.mark[g] = kFreeMark;
  cluster_sync();
  for (int b = cta * 32 + warp; b < p.B; b += kPlanCtas * 32) {
    const int n = pages_len(p.lens, b, p.max_pages, p.page_shift), np = (n >> p.page_shift) + ((n & psm) != 0);
    for (int t = lane; t < np; t += 32) {
      const int page = __ldg(p.table + (long long)b * p.max_pages + t);
      if (pages_ok(page, p.num_pages)) p.mark[page] = page;
    }
  }
  cluster_sync();
  const int g0 = plan_begin(p.num_pages, cta), g1 = plan_begin(p.num_pages, cta + 1);
  auto used = [&](int g) { return g < g1 && __ldcg(p.mark + g) != kFreeMark; };
  int n = 0, total;
  for (int at = g0; at < g1; at += kPlanThreads) {
    block_rank(used(at + threadIdx.x), sm, &total);
    n += total;
  }
  if (threadIdx.x == 0) p.counts[cta] = n;
  cluster_sync();
  int live;
  plan_before(p.counts, cta, &live);
  int holes = 0, moves = 0;
  for (int at = g0; at < g1; at += kPlanThreads) {
    const int g = at + threadIdx.x;
    const bool u = used(g);
    block_rank(g < g1 && g < live && !u, sm, &total);
    holes += total;
    block_rank(g >= live && u, sm, &total);
    moves += total;
  }
  if (threadIdx.x == 0) {
    p.counts[kPlanCtas + cta] = holes;
    p.counts[2 * kPlanCtas + cta] = moves;
  }
  cluster_sync();
  int all_moves;
  int h = plan_before(p.counts + kPlanCtas, cta, &total), m = plan_before(p.counts + 2 * kPlanCtas, cta, &all_moves);
  for (int at = g0; at < g1; at += kPlanThreads) {
    const int g = at + threadIdx.x;
    const bool u = used(g);
    const bool hole = g < g1 && g < live && !u, move = g >= live && u;
    int k = h + block_rank(hole, sm, &total);
    if (hole) p.dst[k] = g;
    h += total;
    k = m + block_rank(move, sm, &total);
    if (move) p.src[k] = g;
    m += total;
  }
  if (tid == 0) {
    *p.n_live = live;
    *p.count = all_moves;
  }
  cluster_sync();
  for (int k = tid; k < all_moves; k += threads) p.mark[__ldcg(p.src + k)] = __ldcg(p.dst + k);
  cluster_sync();
  for (int b = cta * 32 + warp; b < p.B; b += kPlanCtas * 32) {
    const int len = pages_len(p.lens, b, p.max_pages, p.page_shift), np = (len >> p.page_shift) + ((len & psm) != 0);
    const int32_t* from = p.table + (long long)b * p.max_pages;
    int32_t* to = p.table_out + (long long)b * p.max_pages;
    for (int t = lane; t < p.max_pages; t += 32) {
      int page = t < np ? __ldg(from + t) : -1;
      if (page >= 0 && page < p.num_pages) page = __ldcg(p.mark + page);
      to[t] = page;
    }
  }
}

// Copies pages src[k] -> dst[k], k < *count, of every pool (blockIdx.y); no dst is a src.  A block
// moves 16 KB at a time, four vectors a thread, loaded before the first is stored: a part of a
// large page, or several small ones.
constexpr int kCopyBytes = 16384, kCopyThreads = 256;

template <typename T>
__device__ __forceinline__ void copy_pool(uint8_t* base, unsigned bytes, int n, const int32_t* src, const int32_t* dst) {
  constexpr unsigned kVec = kCopyBytes / 16;  // vectors of a piece
  const unsigned vpp = bytes / sizeof(T);     // vectors of a page
  const unsigned pieces = (vpp + kVec - 1) / kVec, pages = vpp < kVec ? kVec / vpp : 1;
  const long long items = pages > 1 ? (n + (long long)pages - 1) / pages : (long long)n * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const unsigned k0 = pages > 1 ? (unsigned)(it * pages) : (unsigned)(it / pieces);
    const unsigned v0 = pages > 1 ? 0u : (unsigned)(it - (long long)k0 * pieces) * kVec;
    const unsigned vn = pages > 1 ? min(pages, (unsigned)n - k0) * vpp : min(kVec, vpp - v0);
    T x[4];
    T* to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned v = j * kCopyThreads + threadIdx.x;
      to[j] = nullptr;
      if (v < vn) {
        const unsigned k = pages > 1 ? v / vpp : 0u, in = pages > 1 ? v - k * vpp : v0 + v;
        const long long from = __ldg(src + k0 + k), at = __ldg(dst + k0 + k);
        x[j] = __ldcs(reinterpret_cast<const T*>(base) + from * vpp + in);
        to[j] = reinterpret_cast<T*>(base) + at * vpp + in;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (to[j]) __stcs(to[j], x[j]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PoolList pools,
                                                                  const int32_t* src, const int32_t* dst,
                                                                  const int32_t* count) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = *count;
  uint8_t* base = pools.base[blockIdx.y];
  const unsigned bytes = pools.bytes[blockIdx.y];
  const unsigned long long mis = reinterpret_cast<uintptr_t>(base) | bytes;
  if ((mis & 15) == 0) copy_pool<uint4>(base, bytes, n, src, dst);
  else if ((mis & 3) == 0) copy_pool<uint32_t>(base, bytes, n, src, dst);
  else copy_pool<uint8_t>(base, bytes, n, src, dst);
}

}  // namespace fa

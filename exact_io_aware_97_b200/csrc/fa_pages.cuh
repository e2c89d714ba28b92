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
// change: one kernel plans (a memset and four small kernels, with the copies, took 26 us on 16 prompts
// forked into 64 sequences, this one and the copies 20 us), one copies.
#pragma once

#include "fa_device.cuh"

namespace fa {

constexpr int kMaxPools = 128, kMaxLaunches = 32;  // pools of a launch, launches
constexpr int kFreeMark = 0x7FFFFFFF;

struct PoolList {
  uint8_t* base[kMaxPools];
  unsigned vpp[kMaxPools];     // vectors of a page
  unsigned pages[kMaxPools];   // whole pages of an item, or 0
  unsigned pieces[kMaxPools];  // else items of a page
  uint8_t vec[kMaxPools];      // bytes of a vector: 16, 4 or 1, what the pages' alignment allows
  int n, bulk;                 // pools; the first `bulk` of them have pages for bulk copies
};

struct ForkParams {
  const int32_t *table, *lens, *parent;
  int32_t *table_out, *lens_out, *free_pages, *n_free;
  int32_t *mark;          // [num_pages]
  int32_t *rank;          // [R]: number of the copy that row i needs, or -1
  int32_t *src, *dst;     // [R]: the copies
  int32_t *count;         // number of copies
  int32_t *tickets;       // [kMaxLaunches]: next piece to copy, for each launch of the copies
  int32_t *counts;        // per CTA of the planning cluster
  int B, R, max_pages, page_shift, num_pages;
};

struct CompactParams {
  const int32_t *table, *lens;
  int32_t *table_out, *n_live;
  int32_t *mark;       // [num_pages]
  int32_t *src, *dst;  // [num_pages / 2 + 1]
  int32_t *count, *counts, *tickets;
  int B, max_pages, page_shift, num_pages;
};

// Length of a sequence, or 0 (recorded) for one that the table cannot hold.
__device__ __forceinline__ int pages_len(const int32_t* lens, int b, int max_pages, int page_shift) {
  const int n = load_in(lens + b);
  if (n < 0 || (long long)n > (long long)max_pages << page_shift) {
    atomicOr(&g_error_word, kErrBadSeqlens);
    return 0;
  }
  return n;
}

__device__ __forceinline__ int fork_len(const ForkParams& p, int i, int* parent) {
  const int b = load_in(p.parent + i);
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
  return load_in(p.table + (long long)b * p.max_pages + (n >> p.page_shift));
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  __shared__ int sm[32];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = cta * kPlanThreads + threadIdx.x, threads = kPlanCtas * kPlanThreads;
  const int psm = (1 << p.page_shift) - 1;
  grid_wait();
  // the copies' blocks may come to the idle SMs now; they wait for this kernel's end
  grid_release();
  if (tid < kMaxLaunches) p.tickets[tid] = 0;
  for (int g = tid; g < p.num_pages; g += threads) p.mark[g] = kFreeMark;
  // this thread's first row of the steps after the marks; lookups that fill the cache meanwhile
  const int i0 = plan_begin(p.R, cta), i1 = plan_begin(p.R, cta + 1);
  const int mine_i = i0 + threadIdx.x, mine_tail = mine_i < i1 ? fork_tail(p, mine_i) : -1;
  auto tail = [&](int i) { return i == mine_i ? mine_tail : i < i1 ? fork_tail(p, i) : -1; };
  if (p.R > 0) {
    int b;
    (void)fork_len(p, (cta * 32 + warp) / ((p.max_pages + 127) / 128) % p.R, &b);
  }
  cluster_sync();
  // mark[page]: -1 where some new row holds it full, else the first new row that ends in it; a
  // warp takes 128 entries of a row, all loaded before the first is marked
  const int strips = (p.max_pages + 127) / 128;
  for (long long it = cta * 32 + warp; it < (long long)p.R * strips; it += kPlanCtas * 32) {
    const int i = (int)(it / strips), t0 = (int)(it - (long long)i * strips) * 128 + lane;
    int b;
    const int n = fork_len(p, i, &b), full = n >> p.page_shift, np = full + ((n & psm) != 0);
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      page[j] = t0 + 32 * j < np ? load_in(p.table + (long long)b * p.max_pages + t0 + 32 * j) : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + 32 * j < np && pages_ok(page[j], p.num_pages))
        atomicMin(p.mark + page[j], t0 + 32 * j < full ? -1 : i);
  }
  cluster_sync();
  // count the copies that this CTA's rows need and the free pages in its part of the pool
  auto needs_copy = [&](int i, int page) { return page >= 0 && page < p.num_pages && __ldcg(p.mark + page) != i; };
  const int g0 = plan_begin(p.num_pages, cta), g1 = plan_begin(p.num_pages, cta + 1);
  // (what the first round of each count finds is kept for the ranks below)
  const int mine_g = g0 + threadIdx.x;
  const bool mine_free = mine_g < g1 && __ldcg(p.mark + mine_g) == kFreeMark;
  const bool mine_copy = mine_i < i1 && needs_copy(mine_i, mine_tail);
  int copies, frees, total;
  const int mine_copy_rank = block_rank(mine_copy, sm, &copies), mine_free_rank = block_rank(mine_free, sm, &frees);
  const int first_copies = copies, first_frees = frees;
  for (int at = i0 + kPlanThreads; at < i1; at += kPlanThreads) {
    const int i = at + threadIdx.x;
    block_rank(i < i1 && needs_copy(i, tail(i)), sm, &total);
    copies += total;
  }
  for (int at = g0 + kPlanThreads; at < g1; at += kPlanThreads) {
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
  auto take_copy = [&](int i, int page, bool copy, int k) {
    if (i < i1) p.rank[i] = copy ? k : -1;
    if (copy) p.src[k] = page;
  };
  auto take_free = [&](int g, bool is_free, int k) {
    if (!is_free) return;
    if (k < need) p.dst[k] = g;
    else p.free_pages[k - need] = g;
  };
  take_copy(mine_i, mine_tail, mine_copy, r + mine_copy_rank);
  take_free(mine_g, mine_free, f + mine_free_rank);
  r += first_copies;
  f += first_frees;
  for (int at = i0 + kPlanThreads; at < i1; at += kPlanThreads) {
    const int i = at + threadIdx.x, page = tail(i);
    const bool copy = i < i1 && needs_copy(i, page);
    take_copy(i, page, copy, r + block_rank(copy, sm, &total));
    r += total;
  }
  for (int at = g0 + kPlanThreads; at < g1; at += kPlanThreads) {
    const int g = at + threadIdx.x;
    const bool is_free = g < g1 && __ldcg(p.mark + g) == kFreeMark;
    take_free(g, is_free, f + block_rank(is_free, sm, &total));
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
  for (long long it = cta * 32 + warp; it < (long long)p.R * strips; it += kPlanCtas * 32) {
    const int i = (int)(it / strips), t0 = (int)(it - (long long)i * strips) * 128 + lane;
    const int k = __ldcg(p.rank + i);
    int b;
    int n = fork_len(p, i, &b);
    if (k >= have) n = 0;  // no page was left for it
    const int full = n >> p.page_shift, np = full + ((n & psm) != 0);
    const int32_t* from = p.table + (long long)max(b, 0) * p.max_pages;
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + 32 * j;
      page[j] = t >= np ? -1 : t == full && k >= 0 ? __ldcg(p.dst + k) : load_in(from + t);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + 32 * j < p.max_pages) p.table_out[(long long)i * p.max_pages + t0 + 32 * j] = page[j];
    if (t0 == 0) p.lens_out[i] = n;
  }
}

__global__ void __cluster_dims__(kPlanCtas) __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  __shared__ int sm[32];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = cta * kPlanThreads + threadIdx.x, threads = kPlanCtas * kPlanThreads;
  const int psm = (1 << p.page_shift) - 1;
  grid_wait();
  // the copies' blocks may come to the idle SMs now; they wait for this kernel's end
  grid_release();
  if (tid < kMaxLaunches) p.tickets[tid] = 0;
  for (int g = tid; g < p.num_pages; g += threads) p.mark[g] = kFreeMark;
  cluster_sync();
  const int strips = (p.max_pages + 127) / 128;  // a warp takes 128 entries of a row
  for (long long it = cta * 32 + warp; it < (long long)p.B * strips; it += kPlanCtas * 32) {
    const int b = (int)(it / strips), t0 = (int)(it - (long long)b * strips) * 128 + lane;
    const int n = pages_len(p.lens, b, p.max_pages, p.page_shift), np = (n >> p.page_shift) + ((n & psm) != 0);
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      page[j] = t0 + 32 * j < np ? load_in(p.table + (long long)b * p.max_pages + t0 + 32 * j) : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + 32 * j < np && pages_ok(page[j], p.num_pages)) p.mark[page[j]] = page[j];
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
  for (long long it = cta * 32 + warp; it < (long long)p.B * strips; it += kPlanCtas * 32) {
    const int b = (int)(it / strips), t0 = (int)(it - (long long)b * strips) * 128 + lane;
    const int len = pages_len(p.lens, b, p.max_pages, p.page_shift), np = (len >> p.page_shift) + ((len & psm) != 0);
    int page[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      page[j] = t0 + 32 * j < np ? load_in(p.table + (long long)b * p.max_pages + t0 + 32 * j) : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (page[j] >= 0 && page[j] < p.num_pages) page[j] = __ldcg(p.mark + page[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + 32 * j < p.max_pages) p.table_out[(long long)b * p.max_pages + t0 + 32 * j] = page[j];
  }
}

// Copies pages src[k] -> dst[k], k < *count, of every pool; no dst is a src.
//
// Large pages (the pools before `bulk`) go through shared memory in pieces of up to 16 KB by bulk
// copies, which one thread issues: a ring of six pieces in flight each way per CTA, two CTAs per SM
// (four vectors a thread in registers instead: 189 to 217 us for the 178 us of a compaction that moves
// 543 MB; the copies alone then run at 6.4 TB/s, read and written, of the 6.55 of a plain copy).
// Small pages go in vectors, four a thread, loaded before the first is stored.
constexpr int kCopyVecs = 1024, kCopyThreads = 256;
constexpr int kBulkBytes = 16384, kBulkStages = 6, kCopySmem = kBulkStages * kBulkBytes + 128;

template <typename T>
__device__ __forceinline__ void copy_item(uint8_t* base, unsigned vpp, unsigned pages, unsigned pieces, long long it,
                                          int n, const int32_t* src, const int32_t* dst) {
  const unsigned k0 = pages ? (unsigned)it * pages : (unsigned)(it / pieces);
  const unsigned v0 = pages ? 0u : (unsigned)(it - (long long)k0 * pieces) * kCopyVecs;
  const unsigned vn = pages ? min(pages, (unsigned)n - k0) * vpp : min((unsigned)kCopyVecs, vpp - v0);
  T x[4];
  T* to[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned v = j * kCopyThreads + threadIdx.x;
    to[j] = nullptr;
    if (v < vn) {
      const unsigned k = pages ? v / vpp : 0u, in = pages ? v - k * vpp : v0 + v;
      const long long from = load_in(src + k0 + k), at = load_in(dst + k0 + k);
      x[j] = __ldcs(reinterpret_cast<const T*>(base) + from * vpp + in);
      to[j] = reinterpret_cast<T*>(base) + at * vpp + in;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (to[j]) __stcs(to[j], x[j]);
}

// Walks the items of pools [pool, stop) that fall to this block.
struct CopyWalk {
  int pool, stop;
  long long it, first;  // item; first item of the pool
  __device__ __forceinline__ bool next(const PoolList& pools, int n) {
    for (;; ++pool) {
      if (pool >= stop) return false;
      const unsigned pages = pools.pages[pool];
      const long long items = pages ? ((long long)n + pages - 1) / pages : (long long)n * pools.pieces[pool];
      if (it < first + items) return true;
      first += items;
    }
  }
};

__global__ void __launch_bounds__(kCopyThreads + 32, 2)
    pages_copy_kernel(const __grid_constant__ PoolList pools, const int32_t* src, const int32_t* dst,
                      const int32_t* count, int32_t* next) {
  extern __shared__ uint8_t smem_raw[];
  grid_wait();
  const int n = *count;
  if (threadIdx.x < kCopyThreads) {
    CopyWalk w{pools.bulk, pools.n, blockIdx.x, 0};
    for (; w.next(pools, n); w.it += gridDim.x) {
      const unsigned vpp = pools.vpp[w.pool], pages = pools.pages[w.pool], pieces = pools.pieces[w.pool];
      uint8_t* const base = pools.base[w.pool];
      const long long it = w.it - w.first;
      if (pools.vec[w.pool] == 16) copy_item<uint4>(base, vpp, pages, pieces, it, n, src, dst);
      else if (pools.vec[w.pool] == 4) copy_item<uint32_t>(base, vpp, pages, pieces, it, n, src, dst);
      else copy_item<uint8_t>(base, vpp, pages, pieces, it, n, src, dst);
    }
    return;
  }
  if (threadIdx.x != kCopyThreads) return;
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem_raw + kBulkStages * kBulkBytes);
  for (int s = 0; s < kBulkStages; ++s) mbar_init(full + s, 1);
  fence_barrier_init();
  // Pieces are handed out by a counter (dealt in equal shares, the first CTA was done at 136 us of
  // 185); which CTA copies a piece changes nothing in the result.  The next ticket is drawn while
  // the last one's piece is loaded.
  CopyWalk walk{0, pools.bulk, 0, 0};
  uint8_t* to[kBulkStages];
  unsigned bytes[kBulkStages];
  long long ticket = atomicAdd(next, 1);
  auto load = [&](int slot) {
    bytes[slot] = 0;
    walk.it = ticket;
    if (!walk.next(pools, n)) return;
    ticket = atomicAdd(next, 1);
    const unsigned pieces = pools.pieces[walk.pool];
    const long long it = walk.it - walk.first, k = it / pieces, piece = it - k * pieces;
    const unsigned long long page = (unsigned long long)pools.vpp[walk.pool] * 16;
    uint8_t* const base = pools.base[walk.pool] + piece * kBulkBytes;
    bytes[slot] = (unsigned)min(page - piece * kBulkBytes, (unsigned long long)kBulkBytes);
    to[slot] = base + (unsigned long long)load_in(dst + k) * page;
    mbar_arrive_expect_tx(full + slot, bytes[slot]);
    bulk_load(smem_raw + slot * kBulkBytes, base + (unsigned long long)load_in(src + k) * page, bytes[slot],
              full + slot);
  };
  // the store of a piece follows its load; the load of the piece five further on follows the store
  // of the one before, once that has read its slot
#pragma unroll
  for (int s = 0; s < kBulkStages - 1; ++s) load(s);
  bool ok = true;
  int late = 0;  // parities of the slots' last fills, once a wait ran out
  for (uint32_t phase = 0; ok; phase ^= 1u) {
#pragma unroll
    for (int s = 0; s < kBulkStages; ++s) {
      if (ok) {
        bulk_wait_group_read0();
        load((s + kBulkStages - 1) % kBulkStages);
        ok = bytes[s] != 0;
        if (ok && !mbar_wait(full + s, phase)) {
          ok = false;
          late = 1 << kBulkStages | (phase ? (1 << kBulkStages) - (1 << s) : (1 << s) - 1);
        }
      }
      if (ok) {
        bulk_store(to[s], smem_raw + s * kBulkBytes, bytes[s]);
        bulk_commit_group();
      }
    }
  }
  if (late)  // leave no copy in flight
#pragma unroll
    for (int s = 0; s < kBulkStages; ++s)
      if (bytes[s] != 0) (void)mbar_wait(full + s, late >> s & 1);
  bulk_wait_group0();
}

}  // namespace fa

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
// Bound by HBM where pages are copied (2 bytes moved a byte) and by launches and one pass over
// the pool's marks where only tables change.
#pragma once

#include "fa_device.cuh"

namespace fa {

constexpr int kMaxPools = 128;
constexpr int kFreeMark = 0x7F7F7F7F;  // what a memset of 0x7F leaves

struct PoolList {
  uint8_t* base[kMaxPools];
  unsigned long long bytes[kMaxPools];  // of one page
  int n;
};

struct ForkParams {
  const int32_t *table, *lens, *parent;
  int32_t *table_out, *lens_out, *free_pages, *n_free;
  int32_t *mark;          // [num_pages]
  int32_t *rank;          // [R]: number of the copy that row i needs, or -1
  int32_t *src, *dst;     // [R]: the copies
  int32_t *count;         // number of copies
  int B, R, max_pages, page_shift, num_pages;
};

struct CompactParams {
  const int32_t *table, *lens;
  int32_t *table_out, *n_live;
  int32_t *mark;       // [num_pages]
  int32_t *src, *dst;  // [num_pages / 2 + 1]
  int32_t *count;
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

// mark[page]: -1 where some new row holds it full, else the first new row that ends in it.
__global__ void __launch_bounds__(256) fork_mark_kernel(const ForkParams p) {
  const int i = blockIdx.x;
  int b;
  const int n = fork_len(p, i, &b);
  const int full = n >> p.page_shift, np = full + ((n & ((1 << p.page_shift) - 1)) != 0);
  for (int t = threadIdx.x; t < np; t += blockDim.x) {
    const int page = __ldg(p.table + (long long)b * p.max_pages + t);
    if (pages_ok(page, p.num_pages)) atomicMin(p.mark + page, t < full ? -1 : i);
  }
}

// Exclusive sum over the 1024 threads of a block of one flag each; total in *total.
__device__ __forceinline__ int block_rank(bool flag, int* sm, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned ballot = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sm[warp] = __popc(ballot);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    const int c = sm[w];
    before += w < warp ? c : 0;
    all += c;
  }
  *total = all;
  return before + __popc(ballot & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(1024) fork_plan_kernel(const ForkParams p) {
  __shared__ int sm[32];
  int need = 0;
  for (int i0 = 0; i0 < p.R; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    bool copy = false;
    int page = -1;
    if (i < p.R) {
      int b;
      const int n = fork_len(p, i, &b);
      if (n & ((1 << p.page_shift) - 1)) {
        page = __ldg(p.table + (long long)b * p.max_pages + (n >> p.page_shift));
        copy = page >= 0 && page < p.num_pages && p.mark[page] != i;
      }
    }
    int total;
    const int r = need + block_rank(copy, sm, &total);
    if (i < p.R) p.rank[i] = copy ? r : -1;
    if (copy) p.src[r] = page;
    need += total;
  }
  int free_pages = 0;
  for (int g0 = 0; g0 < p.num_pages; g0 += 1024) {
    const int g = g0 + threadIdx.x;
    const bool is_free = g < p.num_pages && p.mark[g] == kFreeMark;
    int total;
    const int r = free_pages + block_rank(is_free, sm, &total);
    if (is_free) {
      if (r < need) p.dst[r] = g;
      else p.free_pages[r - need] = g;
    }
    free_pages += total;
  }
  const int left = max(free_pages - need, 0);
  for (int k = left + threadIdx.x; k < p.num_pages; k += 1024) p.free_pages[k] = -1;
  if (threadIdx.x == 0) {
    *p.n_free = left;
    *p.count = min(need, free_pages);
    if (need > free_pages) atomicOr(&g_error_word, kErrNoPages);
  }
}

__global__ void __launch_bounds__(256) fork_write_kernel(const ForkParams p) {
  const int i = blockIdx.x, r = p.rank[i];
  int b;
  int n = fork_len(p, i, &b);
  if (r >= 0 && r >= *p.count) n = 0;  // no page was left for it
  const int full = n >> p.page_shift, np = full + ((n & ((1 << p.page_shift) - 1)) != 0);
  for (int t = threadIdx.x; t < p.max_pages; t += blockDim.x) {
    int page = -1;
    if (t < np) page = (t == full && r >= 0) ? p.dst[r] : __ldg(p.table + (long long)b * p.max_pages + t);
    p.table_out[(long long)i * p.max_pages + t] = page;
  }
  if (threadIdx.x == 0) p.lens_out[i] = n;
}

__global__ void __launch_bounds__(256) compact_mark_kernel(const CompactParams p) {
  const int b = blockIdx.x;
  const int n = pages_len(p.lens, b, p.max_pages, p.page_shift);
  const int np = (n + (1 << p.page_shift) - 1) >> p.page_shift;
  for (int t = threadIdx.x; t < np; t += blockDim.x) {
    const int page = __ldg(p.table + (long long)b * p.max_pages + t);
    if (pages_ok(page, p.num_pages)) p.mark[page] = page;
  }
}

__global__ void __launch_bounds__(1024) compact_plan_kernel(const CompactParams p) {
  __shared__ int sm[32];
  int live = 0;
  for (int g0 = 0; g0 < p.num_pages; g0 += 1024) {
    const int g = g0 + threadIdx.x;
    int total;
    block_rank(g < p.num_pages && p.mark[g] != kFreeMark, sm, &total);
    live += total;
  }
  int holes = 0, moves = 0;
  for (int g0 = 0; g0 < p.num_pages; g0 += 1024) {
    const int g = g0 + threadIdx.x;
    const bool used = g < p.num_pages && p.mark[g] != kFreeMark;
    const bool hole = g < live && !used, move = g >= live && used;
    int total;
    int r = holes + block_rank(hole, sm, &total);
    if (hole) p.dst[r] = g;
    holes += total;
    r = moves + block_rank(move, sm, &total);
    if (move) p.src[r] = g;
    moves += total;
  }
  __syncthreads();  // moves == holes: both count the pages in use past `live`
  for (int k = threadIdx.x; k < moves; k += 1024) p.mark[p.src[k]] = p.dst[k];
  if (threadIdx.x == 0) {
    *p.n_live = live;
    *p.count = moves;
  }
}

__global__ void __launch_bounds__(256) compact_write_kernel(const CompactParams p) {
  const int b = blockIdx.x;
  const int n = pages_len(p.lens, b, p.max_pages, p.page_shift);
  const int np = (n + (1 << p.page_shift) - 1) >> p.page_shift;
  for (int t = threadIdx.x; t < p.max_pages; t += blockDim.x) {
    int page = -1;
    if (t < np) {
      page = __ldg(p.table + (long long)b * p.max_pages + t);
      if (page >= 0 && page < p.num_pages) page = p.mark[page];
    }
    p.table_out[(long long)b * p.max_pages + t] = page;
  }
}

// Copies pages src[k] -> dst[k], k < *count, of every pool.  No dst is a src.
template <typename T>
__device__ __forceinline__ void copy_piece(const uint8_t* s, uint8_t* d, unsigned long long from,
                                           unsigned long long to) {
  for (unsigned long long at = from + threadIdx.x * sizeof(T); at < to; at += blockDim.x * sizeof(T))
    *reinterpret_cast<T*>(d + at) = *reinterpret_cast<const T*>(s + at);
}

__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ PoolList pools, const int32_t* src,
                                                         const int32_t* dst, const int32_t* count) {
  const int n = *count;
  const long long items = (long long)n * pools.n;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int pool = (int)(it / n), k = (int)(it - (long long)pool * n);
    const unsigned long long bytes = pools.bytes[pool];
    const uint8_t* s = pools.base[pool] + (unsigned long long)src[k] * bytes;
    uint8_t* d = pools.base[pool] + (unsigned long long)dst[k] * bytes;
    const unsigned long long mis = reinterpret_cast<uintptr_t>(pools.base[pool]) | bytes;
    if ((mis & 15) == 0) copy_piece<uint4>(s, d, 0, bytes);
    else if ((mis & 3) == 0) copy_piece<uint32_t>(s, d, 0, bytes);
    else copy_piece<uint8_t>(s, d, 0, bytes);
  }
}

}  // namespace fa

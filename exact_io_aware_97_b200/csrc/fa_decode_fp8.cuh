// Decode attention over a paged cache held in e4m3 with a scale for each block of tokens and
// head (sm_100a).
//
// Query token i (of Nq new tokens) and query head h of a sequence of `len` tokens (the new ones
// included) attend to cache rows j <= len - Nq + i of K/V head h / G:
//   t_j = scale * sk_j * (q . k_j),  p_j = e^(t_j - m),  o = sum_j p_j sv_j v_j / sum_j p_j,
// where k_j, v_j are the stored e4m3 values and sk_j, sv_j the scales of their blocks.
//
// Bound by HBM: 2 d bytes per cache row and K/V head are read once (DRAM reads 1.00 times that).
// 8 sequences of 32K rows, 64 query and 8 K/V heads, d = 128: 90 to 92 us, 5.8 to 6.0 TB/s of the 6.55
// that a copy reaches.  What is left is the start (5 us to the first rows), CTAs that end a little
// after the mean although their shares are equal, and the merge (5 us).
//
// Partition.  The Nq * G query rows of one K/V head form tiles of R rows; a unit is (sequence,
// group of K/V heads, tile) and is cut into chunks of cache rows.  A group is four heads (two, one)
// where that divides Hkv and a tile has at most 16 rows: a chunk then reads 4 d bytes side by side
// from each cache row instead of d (8 sequences of 64K rows, 8 heads, d = 128, loads without products:
// 190 us one head at a time, 175 us four).  All units' chunks, one after the other, are dealt to the
// CTAs of one wave in equal contiguous shares, whatever the lengths, so every CTA streams the same
// number of bytes.  A CTA writes the output of units that lie in its share whole; of at most two
// others (its first and its last) it writes partial sums, which fa_decode_fp8_combine_kernel merges
// with the m / l rule.
//
// Products.  e4m3 values are exact in fp16, so K and V are widened in registers (one conversion
// for two values, after ldmatrix) and multiplied on m16n8k16 fp16 tensor-core products with fp32
// sums.  A query row is scaled by a power of two into [1, 2) at its largest element, which keeps
// its bf16 bits in fp16.  The weights p_j sv_j go through fp16 (11 bits; p alone in bf16, as over
// a bf16 cache, has 8) relative to a reference of their own near their largest one, so neither a scale
// far from the others' nor a small p loses bits; p itself is summed in fp32 for l.  A warp takes 16
// consecutive rows at a time, which lie in one scale block: one K and one V scale.
//
// 9 to 16 query rows over 8 sequences of 32K, 8 K/V heads, d = 128: 99 us (5.4 TB/s); 16 of 32K, d = 64: 114 us
// for 16 rows, 239 for 32, 395 for 64 (a floor of 82 us each): latencies and products in registers, at the
// register limit (24 to 152 bytes spilled in each shape).
//
// Up to 8 query rows take fa_decode_fp8_kernel (fa_decode_fp8_narrow.cuh), more than 16 with d = 128
// fa_decode_fp8_tc_kernel (fa_decode_fp8_tc.cuh).  This file has what the three share, the kernel for
// the others and the merge.
#pragma once

#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "fa_decode_sm100.cuh"
#include "fa_device.cuh"

namespace fa {

struct Dec8Params {
  const __nv_bfloat16* q;  // [B, Nq, Hq, D]
  const float* scales[2];  // [num_pages, Hkv, page_size >> sb_shift]
  const int32_t* block_table;
  const int32_t* seqlens;
  __nv_bfloat16* o;
  float* lse;      // [B, Hq, Nq] or null
  float* ws_acc;   // [2 * CTAs][2^hs][R][D]
  float2* ws_ml;   // [2 * CTAs][2^hs][R]: m (base 2), l
  int4* ws_desc;   // [units or CTAs]: the units to merge (see combine)
  int by_unit;     // ws_desc is by unit
  int B, Nq, Hq, Hkv, G, rows, tiles;  // rows = Nq * G, tiles = ceil(rows / R)
  int num_pages, page_shift, sb_shift, max_pages, box;
  int cap;    // rows that the table holds of a sequence
  int units;  // of a sequence: groups of K/V heads * tiles
  int lead;   // positions of a unit before its first chunk
  int hs;     // a unit covers 2^hs K/V heads, a chunk 128 >> hs cache rows of them
  float tau;  // scale * log2(e)
};

constexpr int kDec8Keys = 128;  // cache rows of a chunk, counted over its K/V heads
constexpr int kDec8Whole = 4;   // units of at most this many chunks are not cut (no merge, then, of short tables)
constexpr float kDec8Low = -3e38f;  // references before anything was seen
// A score may be that far (base 2) above its row's reference; only one farther up moves the reference to
// the largest so far, and only then are the lanes' maxima brought together.
constexpr float kDec8Slack = 6.f;

template <int D, int MT, int RG>
struct Dec8WideCfg {
  static constexpr int kRows = 16 * MT * RG;       // R: query rows of a unit
  static constexpr int kWarps = 4 * RG;            // compute warps: 4 slices of 32 rows of the chunk x RG row groups
  // 16-row tiles of the cache that a warp takes at once: two where the registers allow it, for
  // twice the independent chains (one at a time, with two exponentials for each score: 128 us instead
  // of 112 for 8 of 16 rows, 8 sequences of 32K)
  static constexpr int kTiles = MT == 1 ? 2 : 1;
  // A warp with two row tiles needs more registers than its share: the producer then is a warp of
  // a warpgroup of its own, which gives registers up (threads x registers of a CTA: MT = 2, RG = 1:
  // 128 x 208 + 128 x 40 <= 256 x 128; RG = 2: 256 x 224 + 128 x 40 <= 384 x 168).
  static constexpr bool kSplitRegs = MT > 1;
  static constexpr int kComputeRegs = RG == 1 ? 208 : 224;
  static constexpr int kThreads = (kWarps + (kSplitRegs ? 4 : 1)) * 32;
  // per SM: what the registers allow; d = 64 has room for three (8 of 16 rows, 16 sequences of 32K: 118 ->
  // 105 us)
  static constexpr int kCtas = MT == 1 && D == 64 ? 3 : RG == 1 ? 2 : 1;
  static constexpr int kHalf = kDec8Keys * D;       // bytes of K (or V) of a chunk
  static constexpr int kStage = 2 * kHalf;          // also the size of the merge of 16 rows of 4 slices
  static_assert(kStage >= 4 * 16 * D * 4, "a stage holds the sums of 16 query rows of the four slices");
  static constexpr int kStages = D == 128 ? 3 * RG : MT == 1 ? 4 : 6 * RG;
  static constexpr int kQBytes = MT == 1 ? 0 : RG * MT * (D / 16) * 32 * 16;
  static constexpr int kSmem = 1024 + kStages * kStage + kQBytes + RG * 4 * 16 * 8 + kStages * 16 * 4 +
                               2 * kStages * 8;
};

// Position in the sequence of chunks: sequence b, offset u among its units' chunks.
struct Dec8Seg {
  int b, len, chunks;  // sequence, its length and chunks per unit
  int unit;            // group of K/V heads * tiles + tile
  int c0, c1;          // chunks [c0, c1)
};

__device__ __forceinline__ int dec8_len(const Dec8Params& p, int b) {
  return min(max(load_in(p.seqlens + b), 0), p.cap);
}

// Positions count chunks and, before each unit's first, p.lead more that stand for what a unit costs
// on its own (its queries, the start and the end of its pipeline), so that shares of many short units
// take no longer.  Their number is under 2^31 (the host sees to that).
struct Dec8Walk {
  int left, u, b;
  __device__ __forceinline__ bool next(const Dec8Params& p, Dec8Seg& s) {
    while (left > 0) {
      int len;
      for (;; ++b) {  // left > 0: some sequence from b on holds rows
        len = dec8_len(p, b);
        if (len > 0) break;
      }
      s.b = b;
      s.len = len;
      s.chunks = (len - 1 >> 7 - p.hs) + 1;
      const int span = s.chunks + p.lead;
      s.unit = (unsigned)u / (unsigned)span;
      const int from = u - s.unit * span, to = min(span, from + left);
      s.c0 = max(from - p.lead, 0);
      s.c1 = max(to - p.lead, 0);
      left -= to - from;
      u += to - from;
      if (u == span * p.units) {
        ++b;
        u = 0;
      }
      if (s.c0 < s.c1) return true;
    }
    return false;
  }
};

// What the CTAs share out among themselves, in shared memory.
struct Dec8Share {
  int2 scan[32];  // per warp: positions, most positions of a unit
  int b, u, skip[2];
  int end, T, ctas;  // end of this CTA's share (without skip); all positions; CTAs with a share
};

// This CTA's share of all positions, by prefix sums over the sequences; synchronises the CTA.
template <int THREADS>
__device__ __forceinline__ Dec8Walk dec8_share(const Dec8Params& p, Dec8Share& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b_lo = min((int)threadIdx.x * per, p.B), b_hi = min(b_lo + per, p.B);
  auto span_of = [&](int b) {  // positions of one unit of sequence b
    const int n = dec8_len(p, b) + (kDec8Keys >> p.hs) - 1 >> (7 - p.hs);
    return n ? n + p.lead : 0;
  };
  int mine = 0, most = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int n = span_of(b);
    mine += n;
    most = max(most, n);
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) sh.scan[warp] = make_int2(incl, most);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? sh.scan[w].x : 0;
    all += sh.scan[w].x;
    most = max(most, sh.scan[w].y);
  }
  before += incl - mine;
  const int T = all * p.units, ctas = min((int)gridDim.x, T);  // each of these has at least one position
  const bool busy = (int)blockIdx.x < ctas;
  const int quot = busy ? T / ctas : 0, rest = T - quot * ctas;  // share x begins at x T / ctas, rounded down
  int begin = busy ? blockIdx.x * quot + (int)blockIdx.x * rest / ctas : 0;
  int end = busy ? (blockIdx.x + 1) * quot + ((int)blockIdx.x + 1) * rest / ctas : 0;
  // Short sequences: shares begin and end at units (rounded up), nothing is left to merge.
  const bool snap = most <= kDec8Whole + p.lead;
  if (threadIdx.x == 0) {
    sh.skip[0] = sh.skip[1] = 0;  // end == T: no thread finds it
    sh.end = end;
    sh.T = T;
    sh.ctas = ctas;
    if (!p.by_unit) p.ws_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int x = which ? end : begin;
    if (busy && before * p.units <= x && x < (before + mine) * p.units && (which == 0 || snap)) {
      int at = before * p.units, b = b_lo, n;
      for (;; ++b) {
        n = span_of(b) * p.units;
        if (x < at + n) break;
        at += n;
      }
      int skip = 0;
      if (snap) {
        const int c = n / p.units, in = (x - at) % c;
        skip = in ? c - in : 0;
      }
      sh.skip[which] = skip;
      if (which == 0) {
        const bool over = x - at + skip == n;  // on to the next sequence that has rows
        sh.b = b + over;
        sh.u = over ? 0 : x - at + skip;
      }
    }
  }
  __syncthreads();
  if (busy) {
    begin += sh.skip[0];
    end += sh.skip[1];
  }
  return Dec8Walk{end - begin, begin < end ? sh.u : 0, begin < end ? sh.b : 0};
}

// One thread, after a segment: a unit that begins here is described for the merge, if it has to be.
__device__ __forceinline__ void dec8_describe(const Dec8Params& p, const Dec8Seg& seg, const Dec8Share& sh, int group,
                                              int tile, bool whole) {
  if (seg.c0 != 0 || (whole && !p.by_unit)) return;
  // the parts after this one: the CTAs whose shares begin before the unit ends
  int parts = 0;
  if (!whole) {
    // x T / ctas < stop, rounded down or not, is x < stop ctas / T, rounded up
    const long long stop = sh.end + sh.skip[1] + (seg.chunks - seg.c1);
    parts = (int)((stop * sh.ctas + sh.T - 1) / sh.T) - (int)blockIdx.x;
  }
  p.ws_desc[p.by_unit ? seg.b * p.units + seg.unit : blockIdx.x] =
      make_int4(parts | (int)blockIdx.x << 16, seg.b, group, tile);
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 bytes to two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Byte offset of the 16-byte unit `unit` of row `row` in a tile of D-byte rows stored by TMA with
// the 128-byte (D = 128) or 64-byte (D = 64) swizzle.
template <int D>
__device__ __forceinline__ uint32_t dec8_offset(int row, int unit) {
  return row * D + ((D == 128 ? unit ^ (row & 7) : unit ^ ((row >> 1) & 3)) << 4);
}

// V codes of a tile's rows [j0, j0 + 16) that some query does not see (`vs`: the first of them in
// shared memory).  Rows past the end may hold anything and become zeros (by every warp that reads the tile,
// before its own reads; none of them looks at such a row otherwise).  Returns whether a row before the end
// holds a NaN code.
template <int D>
__device__ __noinline__ bool dec8_clean_v(uint8_t* vs, int j0, int len) {
  constexpr int KS = D / 16, n = 16;
  uint32_t nan = 0;
  for (int u = threadIdx.x & 31; u < n * KS; u += 32) {
    uint4* at = reinterpret_cast<uint4*>(vs + u * 16);
    if (j0 + u / KS >= len) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 w = *at;
      nan |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
             ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
    }
  }
  __syncwarp();
  return __any_sync(0xffffffffu, (nan & 0x80808080u) != 0u);
}

// A NaN code may be for some queries only, but 0 * NaN would reach the others: it goes straight
// into the sums of those that see its row (dec8_nan_v), and becomes a zero code (dec8_zero_v).  Rare, so
// calls.
template <int D, int MT>
__device__ __noinline__ void dec8_nan_v(const uint8_t* vs, int j0, int len, const int (&limit)[MT][2],
                                        float (&acc)[MT][D / 8][4]) {
  constexpr int n = 16;
  const int lane = threadIdx.x & 31, tig = lane & 3;
  for (int r = 0; r < n && j0 + r < len; ++r)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(vs + dec8_offset<D>(r, k) + 4 * tig);
#pragma unroll
      for (int x = 0; x < 4; ++x)  // columns 16 k + 4 tig + x
        if (((w >> (8 * x)) & 0x7Fu) == 0x7Fu)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr)
              if (j0 + r < limit[mt][hr]) acc[mt][2 * k + (x & 1)][2 * hr + (x >> 1)] = __uint_as_float(0x7FC00000u);
    }
  __syncwarp();
}

template <int D>
__device__ __noinline__ void dec8_zero_v(uint8_t* vs) {
  for (int u = threadIdx.x & 31; u < 16 * D; u += 32)
    if ((vs[u] & 0x7Fu) == 0x7Fu) vs[u] = 0;
  __syncwarp();
}

// The producer warp's part.  Lanes 0..15: (K or V, K/V head, 16-row tile of the chunk), in the order of
// the warps that take them.  Each fetches the scale of its tile, and the first head's lanes at the head
// of a page's rows the box of them, all heads at once; tiles past the end are left out.  The table
// entry of the next chunk is loaded while this one is issued.
template <int D, int NS>
__device__ __forceinline__ void dec8_produce(const CUtensorMap& tmK, const CUtensorMap& tmV, const Dec8Params& p,
                                             Dec8Walk walk, uint8_t* ring, float* sm_scale, uint64_t* full,
                                             uint64_t* empty) {
  constexpr int kHalf = kDec8Keys * D, kStage = 2 * kHalf;
  const int lane = threadIdx.x & 31;
  if (lane >= 16) return;
  const int which = lane >> 3, sub = lane & 7;
  const uint64_t pol = policy_evict_first();
  const int psm = (1 << p.page_shift) - 1, nb_shift = p.page_shift - p.sb_shift;
  const int chunk = kDec8Keys >> p.hs;
  const int headi = (sub >> 1) >> (2 - p.hs);
  const int ro = 16 * (2 * ((sub >> 1) & ((4 >> p.hs) - 1)) + (sub & 1));  // first row in the chunk
  const bool leads = headi == 0 && ro % p.box == 0;
  Dec8Seg seg;
  int slot = 0;
  uint32_t phase = 1;  // of the slot's release: the first round finds it free
  bool ok = true;
  while (ok && walk.next(p, seg)) {
    const int kvh0 = (seg.unit / p.tiles) << p.hs;
    const int32_t* bt = p.block_table + (long long)seg.b * p.max_pages;
    int tok = seg.c0 * chunk + ro;
    int page_next = tok < seg.len ? load_in(bt + (tok >> p.page_shift)) : 0;
    for (int c = seg.c0; c < seg.c1; ++c, tok += chunk) {
      int page = page_next;
      const bool here = tok < seg.len;
      if (c + 1 < seg.c1 && tok + chunk < seg.len) page_next = load_in(bt + ((tok + chunk) >> p.page_shift));
      if (page < 0 || page >= p.num_pages) {
        atomicOr(&g_error_word, kErrBadPage);
        page = 0;
      }
      ok = __all_sync(0xffffu, mbar_wait(empty + slot, phase));
      if (!ok) break;
      uint8_t* st = ring + slot * kStage;
      if (lane == 0) {
        const int rows = min(chunk, (seg.len - c * chunk + p.box - 1) / p.box * p.box);
        mbar_arrive_expect_tx(full + slot, 2 * (rows << p.hs) * D);
      }
      __syncwarp(0xffffu);
      const int r = tok & psm;
      if (here) {
        if (leads)
          tma_load_3d_hint(st + which * kHalf + (ro << p.hs) * D, which ? &tmV : &tmK, 0, (page << p.page_shift) + r,
                           kvh0, full + slot, pol);
        const float* src =
            p.scales[which] + (((long long)page * p.Hkv + kvh0 + headi) << nb_shift) + (r >> p.sb_shift);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sm_scale + slot * 16 + lane)), "l"(src)
                     : "memory");
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + slot)) : "memory");
      } else {
        sm_scale[slot * 16 + lane] = 0.f;  // a tile past the end may share a warp's step with one before it
        mbar_arrive(full + slot);
      }
      if (++slot == NS) slot = 0, phase ^= 1u;
    }
  }
  if (!ok)  // a wait ran out: leave no copy in flight (the last fill of each slot)
    for (int s = 0; s < NS; ++s) (void)mbar_wait(full + s, s < slot ? phase ^ 1u : phase);
  // the merge may be launched once every CTA has its last loads under way
  if (lane == 0) grid_release();
}

// Sequences without rows, dealt to the CTAs: o = 0, lse = -inf; thread `tid` of THREADS.
template <int D, int THREADS>
__device__ __forceinline__ void dec8_empty(const Dec8Params& p, int tid) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (dec8_len(p, b) > 0) continue;
    const long long n = (long long)p.Nq * p.Hq;
    for (long long k = tid; k < n * D / 8; k += THREADS)
      reinterpret_cast<uint4*>(p.o)[(long long)b * (n * D / 8) + k] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (long long k = tid; k < n; k += THREADS) p.lse[b * n + k] = -INFINITY;
    if (p.by_unit)
      for (int k = tid; k < p.units; k += THREADS) p.ws_desc[b * p.units + k] = make_int4(0, 0, 0, 0);
  }
}

template <int D, int MT, int RG>
__global__ void __launch_bounds__(Dec8WideCfg<D, MT, RG>::kThreads, Dec8WideCfg<D, MT, RG>::kCtas)
    fa_decode_fp8_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const Dec8Params p) {
  using C = Dec8WideCfg<D, MT, RG>;
  constexpr int NS = C::kStages, KS = D / 16, R = C::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint4* sm_q = reinterpret_cast<uint4*>(ring + NS * C::kStage);
  float2* sm_ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(sm_q) + C::kQBytes);  // [RG][4][16]
  float* sm_scale = reinterpret_cast<float*>(sm_ml + RG * 4 * 16);                           // [NS][2][8]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm_scale + NS * 16);
  uint64_t* empty = full + NS;
  __shared__ Dec8Share share;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, 1 + 16);  // the producer's expect_tx, and sixteen lanes' scales
      mbar_init(empty + s, C::kWarps);
    }
    fence_barrier_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }

  grid_wait();
  Dec8Walk walk = dec8_share<C::kThreads>(p, share);
  Dec8Seg seg;

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------ producer
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == C::kWarps) dec8_produce<D, NS>(tmK, tmV, p, walk, ring, sm_scale, full, empty);
    return;
  }

  // -------------------------------------------------------------- compute warps
  if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kComputeRegs));
  constexpr int KT = C::kTiles;
  const int w4 = warp & 3, rg = warp >> 2;  // (K/V head, 32-row slice of the chunk), row group of the tile
  const int headi = w4 >> (2 - p.hs), slice = w4 & ((4 >> p.hs) - 1), chunk = kDec8Keys >> p.hs;
  // where this warp's two tiles are in a chunk: boxes of p.box rows, each [heads][rows][D]
  int toff[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int ro = 32 * slice + 16 * t, in = ro % p.box;
    toff[t] = ((ro - in) << p.hs) * D + (headi * p.box + in) * D;
  }
  const int g = lane >> 2, tig = lane & 3;
  // ldmatrix addresses of this lane within a tile: row (lane & 7) + 8 * ((lane >> 3) & 1), unit
  // lane >> 4 of a pair of units; the swizzle makes the pair 2 k an exclusive or with 2 k.
  const uint32_t ld_off = dec8_offset<D>((lane & 7) + (lane & 8), lane >> 4);
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;

  dec8_empty<D, C::kWarps * 32>(p, threadIdx.x);

  while (walk.next(p, seg)) {
    const int group = seg.unit / p.tiles, tile = seg.unit - group * p.tiles;
    const int kvh = (group << p.hs) + headi;
    const int row0 = tile * R + rg * 16 * MT;  // first query row of this warp
    // rows [16 mt + g + 8 hr]: query token and head, how many cache rows it sees, its factor
    int limit[MT][2];
    float fac[MT][2];
    uint32_t qa[MT == 1 ? KS : 1][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int row = row0 + 16 * mt + g + 8 * hr;
        const bool in = row < p.rows;
        const int i = in ? row / p.G : 0, h = kvh * p.G + (in ? row - i * p.G : 0);
        limit[mt][hr] = in ? seg.len - p.Nq + 1 + i : seg.len;
        const uint2* src =
            reinterpret_cast<const uint2*>(p.q + (((long long)seg.b * p.Nq + i) * p.Hq + h) * D) + tig;
        uint2 x[KS];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          x[k] = in ? load_in(src + 4 * k) : make_uint2(0u, 0u);
          top = max(max(top, max((x[k].x << 16) & 0x7FFF0000u, x[k].x & 0x7FFF0000u)),
                    max((x[k].y << 16) & 0x7FFF0000u, x[k].y & 0x7FFF0000u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with e the exponent of the largest element (0 for a zero row or one that is not finite)
        const int be = (top == 0u || top >= 0x7F800000u) ? 127 : max((int)(top >> 23), 1);
        const float down = be >= 254 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)(254 - be) << 23);
        fac[mt][hr] = p.tau * __uint_as_float((uint32_t)be << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint32_t lo = pack_f16x2(__uint_as_float(x[k].x << 16) * down,
                                         __uint_as_float(x[k].x & 0xFFFF0000u) * down);
          const uint32_t hi = pack_f16x2(__uint_as_float(x[k].y << 16) * down,
                                         __uint_as_float(x[k].y & 0xFFFF0000u) * down);
          if constexpr (MT == 1) {
            qa[k][hr] = lo;      // A fragment: row g + 8 hr, columns 16 k + 4 tig + 0, 1
            qa[k][2 + hr] = hi;  // and + 2, 3 (the order that ldmatrix gives the K bytes in)
          } else if (w4 == 0) {  // MT > 1: one K/V head
            uint32_t* to = reinterpret_cast<uint32_t*>(sm_q + ((rg * MT + mt) * KS + k) * 32 + lane);
            to[hr] = lo;
            to[2 + hr] = hi;
          }
        }
      }
    if constexpr (MT > 1) asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
    // of the whole tile, so that its row groups agree on the cache tiles that they look through
    const int first_limit = seg.len - p.Nq + 1 + tile * R / p.G;
    const bool idle = row0 >= p.rows;  // a row group without rows
    const bool both = RG > 1 && tile * R + 16 * MT < p.rows;  // no row group is
    static_assert(RG <= 2, "two row groups at most");

    float acc[MT][D / 8][4];
    float m_r[MT][2], l_r[MT][2], w_r[MT][2];  // references of t and of t + log2(sv); sum of p
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) acc[mt][n][0] = acc[mt][n][1] = acc[mt][n][2] = acc[mt][n][3] = 0.f;
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        m_r[mt][hr] = w_r[mt][hr] = kDec8Low;
        l_r[mt][hr] = 0.f;
      }
    }

    for (int c = seg.c0; c < seg.c1; ++c) {
      // (after a wait that ran out, recorded, the products go on: whole warps over whatever is there)
      if (ok) ok = mbar_wait(full + slot, phase);
      __syncwarp();
      uint8_t* const st = ring + slot * C::kStage;
      const int jw = c * chunk + 32 * slice;
      if (!idle && jw < seg.len) {
#pragma unroll
        for (int t0 = 0; t0 < 2; t0 += KT) {
          const int j0 = jw + 16 * t0;
          if (KT == 1 && j0 >= seg.len) break;
          const bool partly = j0 + 16 * KT > first_limit;  // rows past the end, or that some query does not see
          if (partly) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              uint8_t* const vs = st + C::kHalf + toff[t0 + kt];
              const bool nan = dec8_clean_v<D>(vs, j0 + 16 * kt, seg.len);
              // the other row group's warp looks at the same tile: neither zeroes a code before both have
              if (!nan) {
                if (RG > 1 && both) asm volatile("bar.sync %0, 64;" ::"r"(2 + w4) : "memory");
                continue;
              }
              // copies, so that the sums themselves stay in registers
              int lim[MT][2];
              float sums[MT][D / 8][4];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                lim[mt][0] = limit[mt][0], lim[mt][1] = limit[mt][1];
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e) sums[mt][n][e] = acc[mt][n][e];
              }
              dec8_nan_v<D, MT>(vs, j0 + 16 * kt, seg.len, lim, sums);
              if (RG > 1 && both) asm volatile("bar.sync %0, 64;" ::"r"(2 + w4) : "memory");
              dec8_zero_v<D>(vs);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[mt][n][e] = sums[mt][n][e];
            }
          }
          const uint32_t base = smem_u32(st) + ld_off;
          float sc[MT][2 * KT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2 * KT; ++n) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; k += 2)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              // matrices: rows 0..7 and 8..15 of the tile, units k and k + 1
              uint32_t w[4], b0, b1;
              ldsm_x4((base + toff[t0 + kt]) ^ (k << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                e4m3x4_to_f16(w[x], b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  if constexpr (MT == 1) {
                    mma_f16_16816(sc[0][2 * kt + (x & 1)], qa[k + (x >> 1)], b0, b1);
                  } else {
                    const uint4 a4 = sm_q[((rg * MT + mt) * KS + k + (x >> 1)) * 32 + lane];
                    const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w};
                    mma_f16_16816(sc[mt][2 * kt + (x & 1)], a, b0, b1);
                  }
                }
              }
            }
          float sk[KT], lsv[KT];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            sk[kt] = sm_scale[slot * 16 + 2 * w4 + t0 + kt];
            lsv[kt] = __log2f(sm_scale[slot * 16 + 8 + 2 * w4 + t0 + kt]);
          }
          // Scores to fp16 weights.  sc is scaled to t = sc * f inside the exponent (f >= 0).
          uint32_t pa[MT][KT][4];
          float mx[MT][2][KT], f[MT][2][KT];
          bool moved = false;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr)
#pragma unroll
              for (int kt = 0; kt < KT; ++kt) {
                float* s0 = &sc[mt][2 * kt][2 * hr];
                float* s1 = &sc[mt][2 * kt + 1][2 * hr];
                if (partly) {
                  const int j = j0 + 16 * kt + 2 * tig, lim = limit[mt][hr];
                  s0[0] = j < lim ? s0[0] : -INFINITY;
                  s0[1] = j + 1 < lim ? s0[1] : -INFINITY;
                  s1[0] = j + 8 < lim ? s1[0] : -INFINITY;
                  s1[1] = j + 9 < lim ? s1[1] : -INFINITY;
                }
                f[mt][hr][kt] = fac[mt][hr] * sk[kt];
                const float x = fmaxf(fmax3(s0[0], s0[1], s1[0]), s1[1]) * f[mt][hr][kt];
                mx[mt][hr][kt] = x;
                moved |= x > m_r[mt][hr] + kDec8Slack || x + lsv[kt] > w_r[mt][hr] + kDec8Slack;
              }
          if (__any_sync(0xffffffffu, moved)) {
            // some score is far above its reference: bring the sums to new ones (NaN never raises one)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float aw[2];
#pragma unroll
              for (int hr = 0; hr < 2; ++hr) {
                float m = m_r[mt][hr], w = w_r[mt][hr];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                  m = fmaxf(m, mx[mt][hr][kt]);
                  w = fmaxf(w, mx[mt][hr][kt] + lsv[kt]);
                }
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                  w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, off));
                }
                l_r[mt][hr] *= ex2_approx(m_r[mt][hr] - m);
                aw[hr] = ex2_approx(w_r[mt][hr] - w);
                m_r[mt][hr] = m;
                w_r[mt][hr] = w;
              }
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                acc[mt][n][0] *= aw[0];
                acc[mt][n][1] *= aw[0];
                acc[mt][n][2] *= aw[1];
                acc[mt][n][3] *= aw[1];
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr)
#pragma unroll
              for (int kt = 0; kt < KT; ++kt) {
                // p = 2^(t - m); the weight is p times cw = sv 2^(m - w), 2^6 at most (the bound keeps
                // 0 * cw at 0 where a scale dwarfs the ones that m came from)
                const float ec = m_r[mt][hr] - w_r[mt][hr] + lsv[kt];
                const float cw = ex2_approx(ec > 120.f ? 120.f : ec);  // NaN stays
                const float ff = f[mt][hr][kt], m = m_r[mt][hr];
                float p0 = ex2_approx(fmaf(sc[mt][2 * kt][2 * hr], ff, -m));
                float p1 = ex2_approx(fmaf(sc[mt][2 * kt][2 * hr + 1], ff, -m));
                float p2 = ex2_approx(fmaf(sc[mt][2 * kt + 1][2 * hr], ff, -m));
                float p3 = ex2_approx(fmaf(sc[mt][2 * kt + 1][2 * hr + 1], ff, -m));
                float w0 = p0 * cw, w1 = p1 * cw, w2 = p2 * cw, w3 = p3 * cw;
                if (partly) {  // a zero or NaN scale says nothing about rows that are not seen
                  const int j = j0 + 16 * kt + 2 * tig, lim = limit[mt][hr];
                  if (j >= lim) p0 = w0 = 0.f;
                  if (j + 1 >= lim) p1 = w1 = 0.f;
                  if (j + 8 >= lim) p2 = w2 = 0.f;
                  if (j + 9 >= lim) p3 = w3 = 0.f;
                }
                l_r[mt][hr] += (p0 + p1) + (p2 + p3);
                pa[mt][kt][hr] = pack_f16x2(w0, w1);
                pa[mt][kt][2 + hr] = pack_f16x2(w2, w3);
              }
#pragma unroll
          for (int k = 0; k < KS; k += 2)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              // transposed: a register holds bytes (2 g, 2 g + 1) of the unit for rows 2 tig and 2 tig + 1
              uint32_t w[4], e0, o0, e1, o1;
              ldsm_x4_t((base + C::kHalf + toff[t0 + kt]) ^ (k << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                e4m3x4_to_f16(__byte_perm(w[2 * x], 0u, 0x3120), e0, o0);
                e4m3x4_to_f16(__byte_perm(w[2 * x + 1], 0u, 0x3120), e1, o1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma_f16_16816(acc[mt][2 * (k + x)], pa[mt][kt], e0, e1);      // columns 16 (k + x) + 2 n
                  mma_f16_16816(acc[mt][2 * (k + x) + 1], pa[mt][kt], o0, o1);  // and + 2 n + 1
                }
              }
            }
        }
      }
      if (c + 1 == seg.c1) break;  // the last slot is kept for the merge
      // The slot is refilled by TMA (the async proxy) once every warp has arrived; the fence
      // orders this warp's generic-proxy reads and writes of it before that.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + slot);
      if (++slot == NS) slot = 0, phase ^= 1u;
    }

    // Merge the slices of each K/V head and row group through the last slot, 16 rows at a time, and
    // write them out.
    const bool whole = seg.c0 == 0 && seg.c1 == seg.chunks;
    const int part = 2 * blockIdx.x + (seg.c0 == 0 ? 1 : 0);
    // final (o, lse) or partial (sums, m, l) results of four columns of a row
    auto put = [&](int kv, int row, int col, float4 A, float M, float L) {
      if (whole) {
        const int i = row / p.G, h = kv * p.G + row - i * p.G;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(p.o + (((long long)seg.b * p.Nq + i) * p.Hq + h) * D + col) =
            make_uint2(pack_bf16x2(A.x * inv, A.y * inv), pack_bf16x2(A.z * inv, A.w * inv));
        if (col == 0 && p.lse)
          p.lse[((long long)seg.b * p.Hq + h) * p.Nq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
      } else {
        const long long at = (((long long)part << p.hs) + kv - (group << p.hs)) * R + row - tile * R;
        *reinterpret_cast<float4*>(p.ws_acc + at * D + col) = A;
        if (col == 0) p.ws_ml[at] = make_float2(M, L);
      }
    };
    if (MT == 1 && RG == 1 && p.hs == 2) {
      // a warp has its K/V head to itself: straight from its registers
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        float l = l_r[0][hr];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = row0 + g + 8 * hr;
        if (row >= p.rows) continue;
        const float e = ex2_approx(w_r[0][hr] - m_r[0][hr]);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          put(kvh, row, 16 * k + 4 * tig,
              make_float4(acc[0][2 * k][2 * hr] * e, acc[0][2 * k + 1][2 * hr] * e, acc[0][2 * k][2 * hr + 1] * e,
                          acc[0][2 * k + 1][2 * hr + 1] * e),
              m_r[0][hr], l);
      }
    } else {
      float* const mg = reinterpret_cast<float*>(ring + slot * C::kStage);
      float2* const ml = sm_ml + rg * 64;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int turn = 0; turn < RG; ++turn) {  // the slot holds one row group's sums
          asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
          if (turn == rg) {
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
              float l = l_r[mt][hr];
              l += __shfl_xor_sync(0xffffffffu, l, 1);
              l += __shfl_xor_sync(0xffffffffu, l, 2);
              // weights so far are relative to 2^w_r: relative to 2^m from here on
              const float e = ex2_approx(w_r[mt][hr] - m_r[mt][hr]);
              if (tig == 0) ml[w4 * 16 + g + 8 * hr] = make_float2(m_r[mt][hr], l);
              float* to = mg + (w4 * 16 + g + 8 * hr) * D + 4 * tig;
#pragma unroll
              for (int k = 0; k < KS; ++k)
                *reinterpret_cast<float4*>(to + 16 * k) =
                    make_float4(acc[mt][2 * k][2 * hr] * e, acc[mt][2 * k + 1][2 * hr] * e,
                                acc[mt][2 * k][2 * hr + 1] * e, acc[mt][2 * k + 1][2 * hr + 1] * e);
            }
          }
          asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
          const int row_at = tile * R + (turn * MT + mt) * 16;  // of the rows now in the slot
          for (int idx = threadIdx.x; idx < (16 << p.hs) * (D / 4); idx += C::kWarps * 32) {
            const int hd = idx / (16 * (D / 4)), r = idx / (D / 4) & 15, col = 4 * (idx % (D / 4));
            const int row = row_at + r, w0 = hd << (2 - p.hs), w1 = (hd + 1) << (2 - p.hs);
            if (row >= p.rows) continue;
            const float2* from = sm_ml + turn * 64 + r;
            float M = kDec8Low, L = 0.f;
            for (int w = w0; w < w1; ++w) M = fmaxf(M, from[w * 16].x);
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = w0; w < w1; ++w) {
              const float e = ex2_approx(from[w * 16].x - M);
              L += e * from[w * 16].y;
              const float4 x = *reinterpret_cast<const float4*>(mg + (w * 16 + r) * D + col);
              A.x += e * x.x;
              A.y += e * x.y;
              A.z += e * x.z;
              A.w += e * x.w;
            }
            put((group << p.hs) + hd, row, col, A, M, L);
          }
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + slot);
    if (++slot == NS) slot = 0, phase ^= 1u;
    if constexpr (MT > 1) asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");  // sm_q is free
    if (threadIdx.x == 0) dec8_describe(p, seg, share, group, tile, whole);
    __syncwarp();
  }
}

// Merges the parts of a unit: part 2 x + 1 of the CTA x it begins in, then the first parts
// 2 (x + 1), 2 (x + 2), ...  blockIdx.x counts units where there are at most as many as CTAs, else
// the CTAs that a unit begins in last (p.by_unit).  WIDE: a block per query row, its warps share
// the parts (few units have many parts each); else a warp per row.
template <int D, int R, bool WIDE>
__global__ void __launch_bounds__(256) fa_decode_fp8_combine_kernel(const Dec8Params p) {
  constexpr int V = D / 32, W = 8;
  __shared__ float sm_l[W], sm_o[W][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  const int4 d = p.ws_desc[blockIdx.x];
  const int parts = d.x & 0xFFFF, x = d.x >> 16;
  if (parts == 0) return;
  const int item = WIDE ? blockIdx.y : blockIdx.y * W + warp;  // row of a tile, over the K/V heads
  const int per = min(p.rows, R), hd = item / per, r = item - hd * per, row = d.w * R + r;
  const bool in = hd < (1 << p.hs) && row < p.rows;
  if (WIDE && !in) return;
  const long long pitch = (long long)R << (1 + p.hs);  // from a CTA's first part to the next one's
  const long long first = ((((long long)2 * x) << p.hs) + hd) * R + r, odd = (long long)R << p.hs;
  float M = kDec8Low, L = 0.f, a[V];
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = 0.f;
  if (in) {
    // every part's maximum first, so that the sums are independent loads
    const int s0 = WIDE ? warp : 0, step = WIDE ? W : 1;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.ws_ml[first + s * pitch + (s ? 0 : odd)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 8
    for (int s = s0; s < parts; s += step) {
      const long long at = first + s * pitch + (s ? 0 : odd);
      const float2 ml = p.ws_ml[at];
      const float d = ml.x - M, e = ex2_approx(d);
      // l of a part whose V scales are far smaller is not: in two halves where the factor is too small for fp32
      const float h = ex2_approx(0.5f * d);
      L += d < -100.f ? ml.y * h * h : e * ml.y;
      if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p.ws_acc + at * D + lane * 4);
        a[0] += e * f.x, a[1] += e * f.y, a[2] += e * f.z, a[3] += e * f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(p.ws_acc + at * D + lane * 2);
        a[0] += e * f.x, a[1] += e * f.y;
      }
    }
  }
  if constexpr (WIDE) {
    if (lane == 0) sm_l[warp] = L;
#pragma unroll
    for (int v = 0; v < V; ++v) sm_o[warp][lane * V + v] = a[v];
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < W; ++w) {
      L += sm_l[w];
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] += sm_o[w][lane * V + v];
    }
  }
  if (!in) return;
  const int i = row / p.G, h = ((d.z << p.hs) + hd) * p.G + row - i * p.G;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat16* to = p.o + (((long long)d.y * p.Nq + i) * p.Hq + h) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(to + v) = pack_bf16x2(a[v] * inv, a[v + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[((long long)d.y * p.Hq + h) * p.Nq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace fa

// Decode attention over an e4m3 paged cache for many query rows: more than 16 of a K/V head (several
// new tokens, large head groups), d = 128 (sm_100a).
//
// The sums of fa_decode_fp8.cuh, with the cache side as M of tcgen05 products, which cost the same for 17
// query rows as for 64.  For a chunk of 128 cache rows and a tile of 64 query rows:
//   S^T [128 rows of K x 64] = K q^T               (A = K's bytes as they are, K-major; q from shared memory)
//   P^T: thread = cache row, its 64 scores to weights
//   O^T [128 columns of V x 64] += V^T P^T         (fp16; A = V widened, read column-major; P from shared memory)
// q goes to e4m3 as the sum of two terms: a row is scaled by a power of two to a largest element in [128,
// 256); hi = e4m3(q), lo = e4m3(q - hi), so hi + lo holds the 8 bits of a bf16 down to 2^-9 of that scale,
// 2^-17 of the row's largest element (both terms into one sum).
// The weights are p sv 2^6 in fp16 (11 bits).  The largest of a row is 2^8 when its reference is set and may
// grow to 2^14.5; only a score that goes beyond raises the reference and rescales the sums, of its block of
// eight rows.  Small weights are in steps of 2^-24, 2^-32 of the largest.  (Weights as two e4m3 terms, with
// V's bytes as they are, took the same time but had steps of 2^-15 of the largest: where one key outweighed
// 32K others by e^11, o was off by 45 %, and by several times bf16's rounding wherever a first token took most
// of the sum.  O is off by 1.65e-3 of its norm on normal data, what bf16 alone gives; it was 1.73e-3.)
// l sums p in fp32.  Both p and w are relative to the one reference, which follows t + log2(sv): p may then be
// as far from 1 as the V scales are from one another (2^-100 .. 2^108 for scales 2^-100 .. 2^100), and
// moves of l by more than fp32's range are taken in two halves.
//
// Warps stay together: whatever lanes do alone ends in a __syncwarp before the next barrier or TMEM
// access, which are for whole warps.
//
// One CTA per SM: TMA producer, MMA issuer, two warps that widen V, four warpgroups that share the query
// rows of every chunk (as two e4m3 terms, two that take the chunks in turn, with 64 scores and 64 sums in
// registers and a merge at each unit's end: 385 us for 40 rows; two that share the rows: 113 us; four in two
// pairs that take the chunks in turn: 118 us; four: 99 us).  Scores, widened V and weights have two buffers,
// so the products of one chunk run under the weights of the next, and the scores of the chunk after that are
// issued before this one's sums (2 % faster than after).  K and V are slots of their own in the ring, since a
// K slot is free as soon as its product is done, a V slot once it is widened and its scales are read.
// (V widened by the warps of the weights: 120 us; by two warps that load 16 bytes, store 32 and so on: 128,
// each load waiting for the stores before it; one row's loads before its first store: 103; one buffer of
// widened V and four chunks in the ring instead of two and three: 104; registers moved between the
// warpgroups: 106 to 136, with spills.)
//
// Bound by the weights: per chunk each warp spends about 170 instructions that do not depend on its
// rows (waits, scales, a vote, loads) and 11 a row, at 51 % of the issue slots; the threads' own accesses take
// 45 % of shared memory's cycles, the products 19 % of the tensor pipe's.  8 sequences of up to 32K rows, 5
// new tokens, 64 query and 8 K/V heads (40 rows): 102 to 104 us for 311 MB, 3.0 TB/s, where the kernel of
// products in registers took 211 us; 8 of 32K: 136 us for 24 rows, 151 for 40, 168 for 64 (a floor of 82; for
// few rows the two warps that widen V are the bound, 2400 cycles a chunk).  For 40 rows the four warpgroups
// have 8, 8, 8 and 16 rows (TMEM is read in blocks of eight), and the chunk waits for the last: an even split
// would save it a quarter of its rows' instructions.
#pragma once

#include "fa_decode_fp8.cuh"

namespace fa {

struct Dec8TcCfg {
  static constexpr int D = 128, kRows = 64;
  static constexpr int kGroups = 4, kWork = 128 * kGroups, kThreads = 128 + kWork;  // warpgroups on the weights
  static constexpr int kSlot = kDec8Keys * D;               // bytes of K (or V) of a chunk
  static constexpr int kSlots = 6, kPairs = kSlots / 2;
  static constexpr int kScales = 8;                         // chunks whose scales are kept (> kPairs)
  static constexpr int kP = kDec8Keys * kRows * 2;          // fp16 weights of a chunk
  static constexpr int kPanel = kDec8Keys * 128, kV = 2 * kPanel;  // 64 columns of V of a chunk in fp16; all
  static constexpr int kQ = kRows * D;                      // hi (and lo) of the query tile
  static constexpr int kColS = 0, kColO = 128, kColOld = 192, kTmemCols = 256;  // S: 2 x 64 columns; O: 64 each
  static constexpr int kRun = 256;                               // chunks that the products add up
  static constexpr int kCols = kRows / kGroups;                  // query rows of a warpgroup, at most
  static constexpr int kOffP = kSlots * kSlot, kOffV = kOffP + 2 * kP, kOffQ = kOffV + 2 * kV;
  static constexpr int kOffMisc = kOffQ + 2 * kQ;
  static constexpr int kSmem = 1024 + kOffMisc + kScales * 64 + kRows * 8 + kRows * 4 + kRows * 16 + 4 * kRows * 4 +
                               64 * 8;
};

// Largest exponent of p sv; the one at a new reference; the weights are p sv 2^6.
constexpr float kTcTop = 8.5f, kTcStart = 2.f, kTcLift = 64.f;

// Instruction descriptor for kind::f16 with fp16 A and B (format code 0), both MN-major, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32_mn(int M, int N) {
  return (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// True for every thread of the warpgroup if it is for one (named barrier `id`, 128 threads).
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred.aligned q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

// Float order as int order (for a maximum over a warp).
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// V codes of a chunk (128-byte rows from `slot`) that some query of the unit does not see: rows past the
// end may hold anything and become zeros; a NaN code would reach every query, so it goes to the queries
// that see its row by hand (sm_nan) and becomes a zero.  Two rows a thread, whole warps.
__device__ __forceinline__ void dec8_tc_clean_v(uint8_t* slot, int first, int j0, int len, int rows,
                                                const int* sm_limit, uint32_t* sm_nan) {
  constexpr int D = Dec8TcCfg::D;
#pragma unroll 1
  for (int row = first; row < kDec8Keys; row += 64) {
    uint8_t* const v = slot + row * D;
    const bool past = j0 + row >= len;
    uint32_t nan = 0;
    uint4* const at16 = reinterpret_cast<uint4*>(v);
    if (past) {
#pragma unroll
      for (int u = 0; u < D / 16; ++u) at16[u ^ (row & 7)] = make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {
        const uint4 y = at16[u ^ (row & 7)];
        nan |= ((y.x & 0x7F7F7F7Fu) + 0x01010101u) | ((y.y & 0x7F7F7F7Fu) + 0x01010101u) |
               ((y.z & 0x7F7F7F7Fu) + 0x01010101u) | ((y.w & 0x7F7F7F7Fu) + 0x01010101u);
      }
    }
    if (!__any_sync(0xffffffffu, (nan & 0x80808080u) != 0u)) continue;
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
      uint8_t* const at = v + (((d >> 4) ^ (row & 7)) << 4) + (d & 15);
      const bool bad = !past && (*at & 0x7Fu) == 0x7Fu;
      if (bad) *at = 0;
      if (__any_sync(0xffffffffu, bad))
#pragma unroll 1
        for (int r = 0; r < rows; ++r)
          if (bad && j0 + row < sm_limit[r]) atomicOr(sm_nan + r * 4 + (d >> 5), 1u << (d & 31));
      __syncwarp();
    }
  }
}

__global__ void __launch_bounds__(Dec8TcCfg::kThreads, 1)
    fa_decode_fp8_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const Dec8Params p) {
  using C = Dec8TcCfg;
  constexpr int D = C::D, R = C::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sm_p = ring + C::kOffP;
  uint8_t* const sm_v = ring + C::kOffV;  // [2 chunks][2][128 rows][64 columns] fp16
  uint8_t* const sm_q = ring + C::kOffQ;
  float* const sm_scale = reinterpret_cast<float*>(ring + C::kOffMisc);        // [kScales][2][8]
  float* const sm_f = sm_scale + C::kScales * 16;             // [R]: factor of a row's scores
  float* const sm_ref = sm_f + R;                             // [R]: minus its reference
  int* const sm_limit = reinterpret_cast<int*>(sm_ref + R);   // [R]
  uint32_t* const sm_nan = reinterpret_cast<uint32_t*>(sm_limit + R);           // [R][4]
  float* const sm_red = reinterpret_cast<float*>(sm_nan + R * 4);               // [2][4][kCols]
  uint64_t* const full = reinterpret_cast<uint64_t*>(sm_red + 4 * R);
  uint64_t* const empty = full + C::kSlots;
  uint64_t* const q_full = empty + C::kSlots;
  uint64_t* const s_full = q_full + 1;    // [2]
  uint64_t* const s_empty = s_full + 2;   // [2]
  uint64_t* const p_full = s_empty + 2;   // [2]
  uint64_t* const p_done = p_full + 2;    // [2]
  uint64_t* const v_full = p_done + 2;    // [2]
  uint64_t* const all_done = v_full + 2;
  __shared__ uint32_t tmem_slot;
  __shared__ Dec8Share share;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(full + s, s & 1 ? 1 + 16 : 1);  // the producer's expect_tx; with V, sixteen lanes' scales
      mbar_init(empty + s, s & 1 ? 2 + C::kWork / 32 : 1);  // V: the warps that widen it, those that take its scales
    }
    mbar_init(q_full, C::kWork / 32);
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + w, 1);
      mbar_init(s_empty + w, C::kWork / 32);
      mbar_init(p_full + w, C::kWork / 32);
      mbar_init(p_done + w, 1);
      mbar_init(v_full + w, 2);
    }
    mbar_init(all_done, 1);
    fence_barrier_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  grid_wait();
  Dec8Walk walk = dec8_share<C::kThreads>(p, share);  // synchronises the CTA
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Dec8Seg seg;

  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      // Lanes 0..15: (K or V, 16-row tile of the chunk), as in fa_decode_fp8_kernel.
      if (lane < 16) {
        const int which = lane >> 3, sub = lane & 7, ro = 16 * sub;
        const uint64_t pol = policy_evict_first();
        const int psm = (1 << p.page_shift) - 1, nb_shift = p.page_shift - p.sb_shift;
        const bool leads = ro % p.box == 0;
        int pair = 0, entry = 0;
        uint32_t phase = 1;
        bool ok = true;
        while (ok && walk.next(p, seg)) {
          const int kvh = seg.unit / p.tiles;
          const int32_t* bt = p.block_table + (long long)seg.b * p.max_pages;
          int tok = seg.c0 * kDec8Keys + ro;
          int page_next = tok < seg.len ? load_in(bt + (tok >> p.page_shift)) : 0;
          for (int c = seg.c0; c < seg.c1; ++c, tok += kDec8Keys) {
            int page = page_next;
            const bool here = tok < seg.len;
            if (c + 1 < seg.c1 && tok + kDec8Keys < seg.len)
              page_next = load_in(bt + ((tok + kDec8Keys) >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
              atomicOr(&g_error_word, kErrBadPage);
              page = 0;
            }
            const int slot = 2 * pair + which;
            ok = __all_sync(0xffffu, mbar_wait(empty + slot, phase));
            if (!ok) break;
            if (sub == 0) {
              const int rows = min(kDec8Keys, (seg.len - c * kDec8Keys + p.box - 1) / p.box * p.box);
              mbar_arrive_expect_tx(full + slot, rows * D);
            }
            __syncwarp(0xffffu);
            const int r = tok & psm;
            float* const to = sm_scale + entry * 16 + lane;
            if (here) {
              if (leads)
                tma_load_3d_hint(ring + slot * C::kSlot + ro * D, which ? &tmV : &tmK, 0, (page << p.page_shift) + r,
                                 kvh, full + slot, pol);
              const float* src = p.scales[which] + (((long long)page * p.Hkv + kvh) << nb_shift) + (r >> p.sb_shift);
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(src) : "memory");
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + 2 * pair + 1))
                           : "memory");
            } else {
              *to = 0.f;
              mbar_arrive(full + 2 * pair + 1);
            }
            if (++pair == C::kPairs) pair = 0, phase ^= 1u;
            entry = (entry + 1) % C::kScales;
          }
        }
        if (!ok)  // a wait ran out: leave no copy in flight (the last fill of each slot)
          for (int s = 0; s < C::kSlots; ++s) (void)mbar_wait(full + s, s >> 1 < pair ? phase ^ 1u : phase);
        if (lane == 0) grid_release();
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idS = idesc_e4m3_f32(128, R), idO = idesc_f16_f32_mn(D, R);
      const uint64_t dRing = smem_desc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t dP = smem_desc_sw128(smem_u32(sm_p), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(sm_v), C::kPanel, 1024);
      const uint64_t dQ = smem_desc_sw128(smem_u32(sm_q), 16, 1024);
      int pair = 0;
      uint32_t kphase = 0, qphase = 0;
      uint32_t n_s = 0, n_p = 0;  // products issued; buffer = the last bit, use of it = the rest
      bool ok = true;
      auto product_s = [&] {
        const uint32_t w = n_s & 1u;
        ok = ok && warp_wait(full + 2 * pair, kphase) && (n_s < 2 || warp_wait(s_empty + w, ((n_s >> 1) - 1) & 1u));
        if (!ok) return;
        tc_fence_after();
        if (elect_one_lane()) {
          const uint64_t a = dRing + (uint64_t)((2 * pair * C::kSlot) >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t)  // hi, lo
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_ss<1>(tmem + C::kColS + w * R, a + (uint64_t)(k * 2), dQ + (uint64_t)((t * C::kQ + k * 32) >> 4), idS,
                        t + k > 0 ? 1u : 0u);
          umma_commit(s_full + w);
          umma_commit(empty + 2 * pair);
        }
        __syncwarp();
        ++n_s;
        if (++pair == C::kPairs) pair = 0, kphase ^= 1u;
      };
      auto product_o = [&](bool first) {
        const uint32_t w = n_p & 1u;
        ok = ok && warp_wait(v_full + w, (n_p >> 1) & 1u) && warp_wait(p_full + w, (n_p >> 1) & 1u);
        if (!ok) return;
        tc_fence_after();
        if (elect_one_lane()) {
          const uint64_t a = dV + (uint64_t)((w * C::kV) >> 4), b = dP + (uint64_t)((w * C::kP) >> 4);
#pragma unroll
          for (int k = 0; k < kDec8Keys / 16; ++k)  // 16 cache rows = 2 KB of either operand
            mma_ss<0>(tmem + C::kColO, a + (uint64_t)(k * 128), b + (uint64_t)(k * 128), idO,
                      first && k == 0 ? 0u : 1u);
          umma_commit(p_done + w);
        }
        __syncwarp();
        ++n_p;
      };
      while (ok && walk.next(p, seg)) {
        const int n = seg.c1 - seg.c0;
        ok = warp_wait(q_full, qphase);
        qphase ^= 1u;
        if (ok) product_s();
        if (ok && n > 1) product_s();
        for (int k = 0; k < n && ok; ++k) {
          if (k + 2 < n) product_s();
          product_o(k % C::kRun == 0);
        }
      }
      umma_commit_elect(all_done);  // nothing is in flight when the columns are given back
      (void)warp_wait(all_done, 0);
    } else {
      // ------------------------------------------------------------ V to fp16: two rows a thread
      const int first = threadIdx.x - 64;
      int pair = 0;
      uint32_t phase = 0, qphase = 0, n = 0;
      bool ok = true;
      while (ok && walk.next(p, seg)) {
        ok = warp_wait(q_full, qphase);  // the tables of the unit's query rows
        qphase ^= 1u;
        const int tile = seg.unit % p.tiles, rows = min(R, p.rows - tile * R);
        const int first_limit = seg.len - p.Nq + 1 + (tile * R) / p.G;
        for (int c = seg.c0; c < seg.c1 && ok; ++c, ++n) {
          ok = warp_wait(full + 2 * pair + 1, phase);
          if (!ok) break;
          uint8_t* const slot = ring + (2 * pair + 1) * C::kSlot;
          const bool partly = (c + 1) * kDec8Keys > first_limit;
          if (partly) dec8_tc_clean_v(slot, first, c * kDec8Keys, seg.len, rows, sm_limit, sm_nan);
          const int sw = first & 7;  // of both rows
          // the product that reads the chunk before the last has ended
          ok = n < 2 || warp_wait(p_done + (n & 1u), ((n >> 1) - 1) & 1u);
          if (!ok) break;
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int row = first + 64 * t;
            uint4 y[D / 16];  // (all of a row before the first store, which might be to where the next load is from)
#pragma unroll
            for (int u = 0; u < D / 16; ++u) y[u] = *reinterpret_cast<const uint4*>(slot + row * D + ((u ^ sw) << 4));
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {  // 16 columns: two units of 8 of panel u / 4
              uint4 h0, h1;
              e4m3x4_to_f16(y[u].x, h0.x, h0.y);
              e4m3x4_to_f16(y[u].y, h0.z, h0.w);
              e4m3x4_to_f16(y[u].z, h1.x, h1.y);
              e4m3x4_to_f16(y[u].w, h1.z, h1.w);
              uint8_t* const to = sm_v + (n & 1u) * C::kV + (u >> 2) * C::kPanel + row * 128;
              *reinterpret_cast<uint4*>(to + (((u & 3) * 2 ^ sw) << 4)) = h0;
              *reinterpret_cast<uint4*>(to + ((((u & 3) * 2 + 1) ^ sw) << 4)) = h1;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_full + (n & 1u));
            mbar_arrive(empty + 2 * pair + 1);
          }
          if (++pair == C::kPairs) pair = 0, phase ^= 1u;
        }
      }
    }
  } else {
    // -------------------------------------------------------------- weights
    const int w = (warp >> 2) - 1, tid = threadIdx.x - 128;  // group; thread among the groups'
    const int row = tid & 127, quarter = row >> 5;           // cache row of a chunk = TMEM lane
    const uint32_t lanes = (uint32_t)quarter << 21;
    float* const red = sm_red + w * 4 * C::kCols;
    int pair = 0, entry = 0;
    uint32_t kphase = 0, n = 0;  // chunks so far: buffer and use as for the MMA issuer
    bool ok = true;

    // sequences without rows: o = 0, lse = -inf
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (dec8_len(p, b) > 0) continue;
      const long long n = (long long)p.Nq * p.Hq;
      for (long long k = tid; k < n * D / 8; k += C::kWork)
        reinterpret_cast<uint4*>(p.o)[(long long)b * (n * D / 8) + k] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (long long k = tid; k < n; k += C::kWork) p.lse[b * n + k] = -INFINITY;
      if (p.by_unit)
        for (int k = tid; k < p.units; k += C::kWork) p.ws_desc[b * p.units + k] = make_int4(0, 0, 0, 0);
    }

    // one arrival for the warp
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    while (walk.next(p, seg)) {
      const int kvh = seg.unit / p.tiles, tile = seg.unit - kvh * p.tiles;
      // this group's query rows: columns [col0, col0 + 8 blocks) of the tile
      const int rows = min(R, p.rows - tile * R), all8 = (rows + 7) >> 3;
      const int col0 = w * all8 / C::kGroups * 8, blocks = (w + 1) * all8 / C::kGroups - w * all8 / C::kGroups;
      const float* const fac = sm_f + col0;
      float* const ref = sm_ref + col0;
      const int* const limit = sm_limit + col0;
      {
        // the query tile: a few threads a row
        constexpr int kPer = C::kWork / R, kVecs = D / 8 / kPer;  // threads of a row; 16-byte vectors of one
        const int r = tid / kPer, part = tid % kPer, qr = tile * R + r;
        const bool in = qr < p.rows;
        const int i = in ? qr / p.G : 0, h = kvh * p.G + (in ? qr - i * p.G : 0);
        const uint4* src =
            reinterpret_cast<const uint4*>(p.q + (((long long)seg.b * p.Nq + i) * p.Hq + h) * D) + part * kVecs;
        uint4 x[kVecs];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          x[k] = in ? load_in(src + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = (&x[k].x)[j];
            top = max(top, max((v << 16) & 0x7FFF0000u, v & 0x7FFF0000u));
          }
        }
#pragma unroll
        for (int off = 1; off < kPer; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const bool finite = top < 0x7F800000u;
        const int be = (top == 0u || !finite) ? 127 : max((int)(top >> 23), 1);
        // 2^(7 - e) in two factors, each a normal number
        const float d0 = __uint_as_float((uint32_t)(127 + (127 - be) / 2) << 23);
        const float d1 = __uint_as_float((uint32_t)(127 + 7 + (127 - be) - (127 - be) / 2) << 23);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t v0 = (&x[k].x)[2 * y], v1 = (&x[k].x)[2 * y + 1];
            const float a[4] = {__uint_as_float(v0 << 16) * d0 * d1, __uint_as_float(v0 & 0xFFFF0000u) * d0 * d1,
                                __uint_as_float(v1 << 16) * d0 * d1, __uint_as_float(v1 & 0xFFFF0000u) * d0 * d1};
            hi[y] = e4m3x4(a[0], a[1], a[2], a[3]);
            uint32_t b0, b1;
            e4m3x4_to_f16(hi[y], b0, b1);
            const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&b0));
            const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&b1));
            lo[y] = e4m3x4(a[0] - f0.x, a[1] - f0.y, a[2] - f1.x, a[3] - f1.y);
          }
          const int byte = (part * kVecs + k) * 8, at = r * D + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 8);
          *reinterpret_cast<uint2*>(sm_q + at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(sm_q + C::kQ + at) = make_uint2(lo[0], lo[1]);
        }
        if (part == 0) {
          // scores are q . k times 2^(e - 7); a row that is not finite makes everything of its own NaN
          sm_f[r] = finite ? p.tau * 0.0078125f * __uint_as_float((uint32_t)be << 23) : __uint_as_float(0x7FC00000u);
          sm_ref[r] = 0.f;
          sm_limit[r] = in ? seg.len - p.Nq + 1 + i : seg.len;
        }
        if (tid < R * 4) sm_nan[tid] = 0u;
      }
      fence_proxy_async_smem();
      __syncwarp();
      asm volatile("bar.sync 1, %0;" ::"n"(C::kWork) : "memory");
      arrive(q_full);

      constexpr int N = C::kCols;
      uint64_t l2[N / 2];  // sums of p, two rows a register pair
#pragma unroll
      for (int r = 0; r < N / 2; ++r) l2[r] = 0;
      const int first_limit = seg.len - p.Nq + 1 + (tile * R) / p.G;

      for (int c = seg.c0; c < seg.c1; ++c, ++n) {
        const uint32_t buf = n & 1u, use = n >> 1;
        // the chunk's scores, scales, and V rows (which may be cleaned here)
        if (ok) ok = mbar_wait(s_full + buf, use & 1u) && mbar_wait(full + 2 * pair + 1, kphase);
        __syncwarp();
        tc_fence_after();
        const int j = c * kDec8Keys + row;
        const float sk = sm_scale[entry * 16 + (row >> 4)];
        float sv = sm_scale[entry * 16 + 8 + (row >> 4)];
        const bool partly = (c + 1) * kDec8Keys > first_limit, fresh = c == seg.c0;
        // (a zero scale weighs nothing; the bound keeps p = 2^(t - reference), up to 2^8.5 / sv, finite)
        float lsv = __log2f(sv);
        lsv = lsv < -100.f ? -100.f : lsv;  // (NaN stays, for the vote)
        float s[N];
#pragma unroll
        for (int b = 0; b < N / 8; ++b)
          if (b < blocks)
            tmem_ld8(tmem + C::kColS + buf * R + col0 + b * 8 + lanes, reinterpret_cast<uint32_t(&)[8]>(s[b * 8]));
        tmem_wait_ld();
        tc_fence_before();
        arrive(s_empty + buf);
        if (lane == 0) mbar_arrive(empty + 2 * pair + 1);  // (the scales have been read)
        // The products' additions drop bits under the last of the sum so far, all downwards: a run of chunks
        // is added to the runs before it, rounded to nearest, and the next one starts at 0.  (One sum over
        // 512K keys was 0.5 % low, over 2M 1.4 %.)
        const int run = c - seg.c0;
        if (run > 0 && run % C::kRun == 0) {
          if (ok) ok = mbar_wait(p_done + (buf ^ 1u), ((n - 1) >> 1) & 1u);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < N / 8; ++b)
            if (b < blocks) {
              float o[8], old[8];
              const uint32_t at = tmem + col0 + b * 8 + lanes;
              tmem_ld8(at + C::kColO, reinterpret_cast<uint32_t(&)[8]>(o));
              tmem_ld8(at + C::kColOld, reinterpret_cast<uint32_t(&)[8]>(old));
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 8; ++x) o[x] = run > C::kRun ? o[x] + old[x] : o[x];
              tmem_st8(at + C::kColOld, reinterpret_cast<uint32_t(&)[8]>(o));
            }
          tmem_wait_st();
        }
        // exponents t - reference, and whether one is past the top
        float most[N / 8];
        bool past_top = false;
        const uint64_t sk2 = f2(sk, sk);
#pragma unroll
        for (int b = 0; b < N / 8; ++b)
          if (b < blocks) {
#pragma unroll
            for (int x = b * 8; x < b * 8 + 8; x += 4) {
              const float4 f = *reinterpret_cast<const float4*>(fac + x), m = *reinterpret_cast<const float4*>(ref + x);
              f2_split(f2_fma(f2(s[x], s[x + 1]), f2_mul(f2(f.x, f.y), sk2), f2(m.x, m.y)), s[x], s[x + 1]);
              f2_split(f2_fma(f2(s[x + 2], s[x + 3]), f2_mul(f2(f.z, f.w), sk2), f2(m.z, m.w)), s[x + 2], s[x + 3]);
            }
          }
        if (partly) {
#pragma unroll
          for (int x = 0; x < N; ++x)
            if (j >= limit[x < blocks * 8 ? x : 0]) s[x] = -INFINITY;
        }
#pragma unroll
        for (int b = 0; b < N / 8; ++b) {
          most[b] = kDec8Low;
          if (b < blocks)
#pragma unroll
            for (int x = b * 8; x < b * 8 + 8; x += 2) most[b] = fmax3(most[b], s[x], s[x + 1]);
          past_top |= !(most[b] + lsv <= kTcTop);
        }
        if (group_any(2 + w, fresh || past_top)) {
          if (__any_sync(0xffffffffu, !(sv < INFINITY))) {
            // (rare) a scale that is not finite makes NaN of what sees its rows, and of nothing else
            const bool bad = !(sv < INFINITY);
            if (w == 0)
#pragma unroll 1
              for (int r = 0; r < rows; ++r)
                if (bad && j < sm_limit[r])
                  for (int k = 0; k < 4; ++k) atomicOr(sm_nan + r * 4 + k, 0xFFFFFFFFu);
            if (bad) sv = 0.f, lsv = -100.f;
            __syncwarp();
          }
          // new references: the largest exponent of each row over the group's threads; a warp looks
          // at the blocks in which it has one past the top
#pragma unroll
          for (int b = 0; b < N / 8; ++b)
            if (b < blocks) {
              float m = kDec8Low;  // lane x < 8: of row 8 b + x
              if (__any_sync(0xffffffffu, fresh || most[b] + lsv > kTcTop))
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const float v = s[b * 8 + x] + lsv;
                  const int i = __reduce_max_sync(0xffffffffu, v == v ? ordered(v) : ordered(-INFINITY));
                  if (lane == x) m = unordered(i);
                }
              if (lane < 8) red[quarter * N + b * 8 + lane] = m;
            }
          __syncwarp();
          asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
          // the sums so far move to the new references (after the last product into them)
          if (!fresh && ok) ok = mbar_wait(p_done + (buf ^ 1u), ((n - 1) >> 1) & 1u);
          __syncwarp();
          tc_fence_after();
          const float least = fresh ? -INFINITY : kTcTop;  // rows at most there keep their reference
#pragma unroll
          for (int b = 0; b < N / 8; ++b)
            if (b < blocks) {
              float up[8], any = -INFINITY;
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int r = b * 8 + x;
                up[x] = fmaxf(fmax3(red[r], red[N + r], red[2 * N + r]), red[3 * N + r]);
                any = fmaxf(any, up[x]);
              }
              if (any <= least) continue;
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int r = b * 8 + x;
                up[x] = up[x] > least ? up[x] - kTcStart : 0.f;
                s[r] -= up[x];
              }
              if (!fresh) {  // (a first reference may lie anywhere: no factor for sums of 0, which may be infinite)
                // l holds every key whatever its V scale, so a factor too small for fp32 is taken in two halves
                const bool far = any > 100.f;
#pragma unroll
                for (int x = 0; x < 8; x += 2) {
                  const float k = far ? -0.5f : -1.f;
                  const uint64_t down = f2(ex2_approx(k * up[x]), ex2_approx(k * up[x + 1]));
                  uint64_t& l = l2[b * 4 + x / 2];
                  l = f2_mul(l, down);
                  if (far) l = f2_mul(l, down);
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) up[x] = ex2_approx(-up[x]);
                for (int old = 0; old <= (run >= C::kRun); ++old) {
                  float o[8];
                  const uint32_t at = tmem + (old ? C::kColOld : C::kColO) + col0 + b * 8 + lanes;
                  tmem_ld8(at, reinterpret_cast<uint32_t(&)[8]>(o));
                  tmem_wait_ld();
#pragma unroll
                  for (int x = 0; x < 8; ++x) o[x] *= up[x];
                  tmem_st8(at, reinterpret_cast<uint32_t(&)[8]>(o));
                }
              }
            }
          tmem_wait_st();
          if (row < blocks * 8) {  // (every thread has used the old references)
            const float m = fmaxf(fmax3(red[row], red[N + row], red[2 * N + row]), red[3 * N + row]);
            if (m > least) ref[row] -= m - kTcStart;
          }
          __syncwarp();
          asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
        }
        // the weights replace those of the chunk before the last once their product is done
        if (n >= 2 && ok) ok = mbar_wait(p_done + buf, (use - 1) & 1u);
        uint8_t* const prow = sm_p + buf * C::kP + row * 128;
        const uint64_t sv2 = f2(sv * kTcLift, sv * kTcLift);
#pragma unroll
        for (int b = 0; b < N / 8; ++b)
          if (b < blocks) {
            uint4 h;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = b * 8 + 2 * x;
              const uint64_t p0 = f2(ex2_approx(s[r]), ex2_approx(s[r + 1]));
              l2[r / 2] = f2_add(l2[r / 2], p0);
              float w0, w1;
              f2_split(f2_mul(p0, sv2), w0, w1);
              (&h.x)[x] = pack_f16x2(w0, w1);
            }
            *reinterpret_cast<uint4*>(prow + ((((col0 >> 3) + b) ^ (row & 7)) << 4)) = h;
          }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(p_full + buf);
        if (++pair == C::kPairs) pair = 0, kphase ^= 1u;
        entry = (entry + 1) % C::kScales;
      }

      // ------------------------------------------------------------ a unit's end
      float l[N];
#pragma unroll
      for (int r = 0; r < N; r += 2) f2_split(l2[r / 2], l[r], l[r + 1]);
      // l of a row over the 128 threads: half of the rows are exchanged between lanes 16 apart, half
      // of the rest between lanes 8 apart, ..., so that lane x ends with the sum of row x (N = 32),
      // or two lanes with halves of it (N = 16)
#pragma unroll
      for (int off = 16, m = N; off > 0; off >>= 1, m = m > 1 ? m >> 1 : 1) {
        const bool upper = (lane & off) != 0;
        if (m == 1) {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
        } else {
#pragma unroll
          for (int r = 0; r < N / 2; ++r)
            if (r < m / 2) {
              const float give = upper ? l[r] : l[r + m / 2], keep = upper ? l[r + m / 2] : l[r];
              l[r] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
      }
      if (lane % (32 / N) == 0) red[quarter * N + lane / (32 / N)] = l[0];
      if (ok) ok = mbar_wait(p_done + ((n - 1) & 1u), ((n - 1) >> 1) & 1u);
      __syncwarp();
      tc_fence_after();
      asm volatile("bar.sync 1, %0;" ::"n"(C::kWork) : "memory");
      const bool whole = seg.c0 == 0 && seg.c1 == seg.chunks;
      const long long part = 2ll * blockIdx.x + (seg.c0 == 0 ? 1 : 0);
#pragma unroll
      for (int b = 0; b < N / 8; ++b)
        if (b < blocks) {
          float sum[8], old[8];
          const uint32_t from = tmem + col0 + b * 8 + lanes;
          tmem_ld8(from + C::kColO, reinterpret_cast<uint32_t(&)[8]>(sum));
          tmem_ld8(from + C::kColOld, reinterpret_cast<uint32_t(&)[8]>(old));
          tmem_wait_ld();
          if (seg.c1 - seg.c0 > C::kRun)
#pragma unroll
            for (int x = 0; x < 8; ++x) sum[x] += old[x];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int r = b * 8 + x, tr = col0 + r, qr = tile * R + tr;
            if (tr >= rows) continue;
            const float L = red[r] + red[N + r] + red[2 * N + r] + red[3 * N + r];
            const float M = L == 0.f ? kDec8Low : -ref[r];  // nothing seen: no reference
            float A = sum[x] * (1.f / kTcLift);
            if ((sm_nan[tr * 4 + (row >> 5)] >> (row & 31)) & 1u) A = __uint_as_float(0x7FC00000u);
            if (whole) {
              const int i = qr / p.G, h = kvh * p.G + qr - i * p.G;
              const float inv = L == 0.f ? 0.f : 1.f / L;
              p.o[(((long long)seg.b * p.Nq + i) * p.Hq + h) * D + row] = __float2bfloat16_rn(A * inv);
              if (row == 0 && p.lse)
                p.lse[((long long)seg.b * p.Hq + h) * p.Nq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
            } else {
              p.ws_acc[(part * R + tr) * D + row] = A;
              if (row == 0) p.ws_ml[part * R + tr] = make_float2(M, L);
            }
          }
        }
      tc_fence_before();
      if (tid == 0) dec8_describe(p, seg, share, kvh, tile, whole);
      __syncwarp();
      asm volatile("bar.sync 1, %0;" ::"n"(C::kWork) : "memory");  // the tables are free for the next unit
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace fa

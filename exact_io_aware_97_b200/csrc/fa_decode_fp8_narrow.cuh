// Decode over the e4m3 paged cache for up to 8 query rows of a K/V head (sm_100a): see
// fa_decode_fp8.cuh for the sharing out of the chunks, the producer, the arithmetic and the merge.
//
// The products are turned round, S^T = K q^T and O^T = V^T P^T: 16 cache rows, or 16 columns of V,
// are the 16 rows of an m16n8k16 product and the query rows its 8 columns, so that 8 query heads of
// a K/V head (or fewer) waste no half of the products, the exponentials and the registers.  P^T
// comes out of the first product with a lane's cache row in its row and goes into the second with
// it in its column: one 8x8 transposition in registers for each half of a tile.  With 8 rows as a
// 16-row operand, 303 instructions of a warp for 16 cache rows and two CTAs per SM, 8 sequences of
// 32K rows took 100 us and, once the power limit has the clock at 1780 MHz, 110 (latencies, not
// HBM, were the bound); so, with 247 instructions and three CTAs per SM, 90, and 92 at 1640 MHz.
// (16 rows this way, as two 8-column operands, spill and are slower than as one 16-row operand.)
#pragma once

#include "fa_decode_fp8.cuh"

namespace fa {

template <int D>
struct Dec8Cfg {
  static constexpr int kRows = 8;                   // query rows of a unit
  static constexpr int kWarps = 4;                  // compute warps
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kCtas = 3;                   // per SM: what the registers allow
  static constexpr int kHalf = kDec8Keys * D;       // bytes of K (or V) of a chunk
  static constexpr int kStage = 2 * kHalf;          // also the size of the merge of four slices
  static_assert(kStage >= 4 * kRows * D * 4, "a stage holds the sums of the query rows of four slices");
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kSmem = 1024 + kStages * kStage + 4 * kRows * 8 + kStages * 16 * 4 + 2 * kStages * 8;
};

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// As dec8_nan_v, with sums acc[u][2 x + e] of column 16 u + 2 g + x and query row 2 tig + e.
template <int D>
__device__ __noinline__ void dec8_nan_vt(uint8_t* vs, int j0, int len, const int (&limit)[2], float (&acc)[D / 16][4]) {
  constexpr int n = 16;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  for (int r = 0; r < n && j0 + r < len; ++r)
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(vs + dec8_offset<D>(r, u) + 2 * g);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (((w >> (8 * x)) & 0x7Fu) == 0x7Fu)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (j0 + r < limit[e]) acc[u][2 * x + e] = __uint_as_float(0x7FC00000u);
    }
  __syncwarp();
  for (int u = lane; u < n * D; u += 32)
    if ((vs[u] & 0x7Fu) == 0x7Fu) vs[u] = 0;
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(Dec8Cfg<D>::kThreads, Dec8Cfg<D>::kCtas)
    fa_decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const Dec8Params p) {
  using C = Dec8Cfg<D>;
  constexpr int NS = C::kStages, KS = D / 16, R = C::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* sm_ml = reinterpret_cast<float2*>(ring + NS * C::kStage);  // [4][R]
  float* sm_scale = reinterpret_cast<float*>(sm_ml + 4 * R);         // [NS][2][8]
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

  if (warp == C::kWarps) {
    dec8_produce<D, NS>(tmK, tmV, p, walk, ring, sm_scale, full, empty);
    return;
  }

  // -------------------------------------------------------------- compute warps
  // (K/V head, 32-row slice of the chunk)
  const int headi = warp >> (2 - p.hs), slice = warp & ((4 >> p.hs) - 1), chunk = kDec8Keys >> p.hs;
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
    const int row0 = tile * R;
    // B fragments of q: row g, columns 16 k + 4 tig + 0, 1 and + 2, 3 (the order that ldmatrix gives
    // the K bytes in)
    uint32_t qb[KS][2];
    int limit[2];  // of rows 2 tig + e: cache rows that they see
    float fac[2];  // factor of their scores
    {
      const int row = row0 + g;
      const bool in = row < p.rows;
      const int i = in ? row / p.G : 0, h = kvh * p.G + (in ? row - i * p.G : 0);
      const uint2* src = reinterpret_cast<const uint2*>(p.q + (((long long)seg.b * p.Nq + i) * p.Hq + h) * D) + tig;
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
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qb[k][0] = pack_f16x2(__uint_as_float(x[k].x << 16) * down, __uint_as_float(x[k].x & 0xFFFF0000u) * down);
        qb[k][1] = pack_f16x2(__uint_as_float(x[k].y << 16) * down, __uint_as_float(x[k].y & 0xFFFF0000u) * down);
      }
      const float f = p.tau * __uint_as_float((uint32_t)be << 23);
      const int lim = in ? seg.len - p.Nq + 1 + i : seg.len;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[e] = __shfl_sync(0xffffffffu, f, (2 * tig + e) * 4);
        limit[e] = __shfl_sync(0xffffffffu, lim, (2 * tig + e) * 4);
      }
    }
    const int first_limit = seg.len - p.Nq + 1 + row0 / p.G;

    float acc[KS][4];  // sums of column 16 u + 2 g + x and row 2 tig + e: [u][2 x + e]
    float m_r[2], l_r[2], w_r[2];  // references of t and of t + log2(sv); sum of p
#pragma unroll
    for (int u = 0; u < KS; ++u) acc[u][0] = acc[u][1] = acc[u][2] = acc[u][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_r[e] = w_r[e] = kDec8Low;
      l_r[e] = 0.f;
    }

    for (int c = seg.c0; c < seg.c1; ++c) {
      // (after a wait that ran out, recorded, the products go on: whole warps over whatever is there)
      if (ok) ok = mbar_wait(full + slot, phase);
      __syncwarp();
      uint8_t* const st = ring + slot * C::kStage;
      const int j0 = c * chunk + 32 * slice;
      if (j0 < seg.len) {
        const bool partly = j0 + 32 > first_limit;  // rows past the end, or that some query does not see
        if (partly) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            uint8_t* const vs = st + C::kHalf + toff[kt];
            if (!dec8_clean_v<D>(vs, j0 + 16 * kt, seg.len)) continue;
            // copies, so that the sums themselves stay in registers
            const int lim[2] = {limit[0], limit[1]};
            float sums[KS][4];
#pragma unroll
            for (int u = 0; u < KS; ++u)
#pragma unroll
              for (int y = 0; y < 4; ++y) sums[u][y] = acc[u][y];
            dec8_nan_vt<D>(vs, j0 + 16 * kt, seg.len, lim, sums);
#pragma unroll
            for (int u = 0; u < KS; ++u)
#pragma unroll
              for (int y = 0; y < 4; ++y) acc[u][y] = sums[u][y];
          }
        }
        const uint32_t base = smem_u32(st) + ld_off;
        // scores of cache row g + 8 y of a tile and query row 2 tig + e: sc[kt][2 y + e]
        float sc[2][4];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) sc[kt][0] = sc[kt][1] = sc[kt][2] = sc[kt][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2)
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            // matrices: rows 0..7 and 8..15 of the tile, units k and k + 1
            uint32_t w[4], a[4];
            ldsm_x4((base + toff[kt]) ^ (k << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              e4m3x4_to_f16(w[2 * x], a[0], a[2]);
              e4m3x4_to_f16(w[2 * x + 1], a[1], a[3]);
              mma_f16_16816(sc[kt], a, qb[k + x][0], qb[k + x][1]);
            }
          }
        // Scores to fp16 weights.  sc is scaled to t = sc * f inside the exponent (f >= 0).
        float lsv[2], f[2][2], mx[2][2];
        bool moved = false;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const float sk = sm_scale[slot * 16 + 2 * warp + kt];
          lsv[kt] = __log2f(sm_scale[slot * 16 + 8 + 2 * warp + kt]);
          if (partly) {
            const int j = j0 + 16 * kt + g;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[kt][e] = j < limit[e] ? sc[kt][e] : -INFINITY;
              sc[kt][2 + e] = j + 8 < limit[e] ? sc[kt][2 + e] : -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[kt][e] = fac[e] * sk;
            const float x = fmaxf(sc[kt][e], sc[kt][2 + e]) * f[kt][e];
            mx[kt][e] = x;
            moved |= x > m_r[e] + kDec8Slack || x + lsv[kt] > w_r[e] + kDec8Slack;
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
          // some score is far above its reference: bring the sums to new ones (NaN never raises one)
          float aw[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmax3(m_r[e], mx[0][e], mx[1][e]);
            float w = fmax3(w_r[e], mx[0][e] + lsv[0], mx[1][e] + lsv[1]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
              w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, off));
            }
            l_r[e] *= ex2_approx(m_r[e] - m);
            aw[e] = ex2_approx(w_r[e] - w);
            m_r[e] = m;
            w_r[e] = w;
          }
#pragma unroll
          for (int u = 0; u < KS; ++u) {
            acc[u][0] *= aw[0];
            acc[u][1] *= aw[1];
            acc[u][2] *= aw[0];
            acc[u][3] *= aw[1];
          }
        }
        uint32_t pb[2][2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // p = 2^(t - m); the weight is p times cw = sv 2^(m - w), 2^6 at most (the bound keeps
            // 0 * cw at 0 where a scale dwarfs the ones that m came from)
            const float ec = m_r[e] - w_r[e] + lsv[kt];
            const float cw = ex2_approx(ec > 120.f ? 120.f : ec);  // NaN stays
            float p0 = ex2_approx(fmaf(sc[kt][e], f[kt][e], -m_r[e]));
            float p1 = ex2_approx(fmaf(sc[kt][2 + e], f[kt][e], -m_r[e]));
            w[e] = p0 * cw;
            w[2 + e] = p1 * cw;
            if (partly) {  // a zero or NaN scale says nothing about rows that are not seen
              const int j = j0 + 16 * kt + g;
              if (j >= limit[e]) p0 = w[e] = 0.f;
              if (j + 8 >= limit[e]) p1 = w[2 + e] = 0.f;
            }
            l_r[e] += p0 + p1;
          }
          pb[kt][0] = transpose_8x8(pack_f16x2(w[0], w[1]));
          pb[kt][1] = transpose_8x8(pack_f16x2(w[2], w[3]));
        }
#pragma unroll
        for (int k = 0; k < KS; k += 2)
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            // transposed: a register holds bytes (2 g, 2 g + 1) of the unit for rows 2 tig and 2 tig + 1
            uint32_t w[4], a[4];
            ldsm_x4_t((base + C::kHalf + toff[kt]) ^ (k << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              e4m3x4_to_f16(__byte_perm(w[2 * x], 0u, 0x3120), a[0], a[1]);
              e4m3x4_to_f16(__byte_perm(w[2 * x + 1], 0u, 0x3120), a[2], a[3]);
              mma_f16_16816(acc[k + x], a, pb[kt][0], pb[kt][1]);
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

    // Merge the slices of each K/V head through the last slot, and write them out.
    const bool whole = seg.c0 == 0 && seg.c1 == seg.chunks;
    const int part = 2 * blockIdx.x + (seg.c0 == 0 ? 1 : 0);
    // final (o, lse) or partial (sums, m, l) results of two or four columns of a row
    auto put = [&](int kv, int row, int col, auto& A, float M, float L) {
      constexpr int V = sizeof(A) / sizeof(float);
      if (whole) {
        const int i = row / p.G, h = kv * p.G + row - i * p.G;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        __nv_bfloat16* to = p.o + (((long long)seg.b * p.Nq + i) * p.Hq + h) * D + col;
#pragma unroll
        for (int v = 0; v < V; v += 2)
          *reinterpret_cast<uint32_t*>(to + v) = pack_bf16x2(A[v] * inv, A[v + 1] * inv);
        if (col == 0 && p.lse)
          p.lse[((long long)seg.b * p.Hq + h) * p.Nq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
      } else {
        const long long at = (((long long)part << p.hs) + kv - (group << p.hs)) * R + row - row0;
        float* to = p.ws_acc + at * D + col;
#pragma unroll
        for (int v = 0; v < V; v += 2) *reinterpret_cast<float2*>(to + v) = make_float2(A[v], A[v + 1]);
        if (col == 0) p.ws_ml[at] = make_float2(M, L);
      }
    };
    float* const mg = reinterpret_cast<float*>(ring + slot * C::kStage);  // [4][R][D]
    if (p.hs < 2) asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_r[e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const int r = 2 * tig + e;
      // weights so far are relative to 2^w_r: relative to 2^m from here on
      const float back = ex2_approx(w_r[e] - m_r[e]);
      if (p.hs == 2) {  // a warp has its K/V head to itself: straight from its registers
        if (row0 + r < p.rows)
#pragma unroll
          for (int u = 0; u < KS; ++u) {
            const float A[2] = {acc[u][e] * back, acc[u][2 + e] * back};
            put(kvh, row0 + r, 16 * u + 2 * g, A, m_r[e], l);
          }
      } else {
        if (g == 0) sm_ml[warp * R + r] = make_float2(m_r[e], l);
#pragma unroll
        for (int u = 0; u < KS; ++u)
          *reinterpret_cast<float2*>(mg + (warp * R + r) * D + 16 * u + 2 * g) =
              make_float2(acc[u][e] * back, acc[u][2 + e] * back);
      }
    }
    if (p.hs < 2) {
      asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
      for (int idx = threadIdx.x; idx < (R << p.hs) * (D / 4); idx += C::kWarps * 32) {
        const int hd = idx / (R * (D / 4)), r = idx / (D / 4) % R, col = 4 * (idx % (D / 4));
        const int w0 = hd << (2 - p.hs), w1 = (hd + 1) << (2 - p.hs);
        if (row0 + r >= p.rows) continue;
        float M = kDec8Low, L = 0.f;
        for (int w = w0; w < w1; ++w) M = fmaxf(M, sm_ml[w * R + r].x);
        float A[4] = {0.f, 0.f, 0.f, 0.f};
        for (int w = w0; w < w1; ++w) {
          const float e = ex2_approx(sm_ml[w * R + r].x - M);
          L += e * sm_ml[w * R + r].y;
          const float4 x = *reinterpret_cast<const float4*>(mg + (w * R + r) * D + col);
          A[0] += e * x.x;
          A[1] += e * x.y;
          A[2] += e * x.z;
          A[3] += e * x.w;
        }
        put((group << p.hs) + hd, row0 + r, col, A, M, L);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + slot);
    if (++slot == NS) slot = 0, phase ^= 1u;
    if (threadIdx.x == 0) dec8_describe(p, seg, share, group, tile, whole);
    __syncwarp();
  }
}

}  // namespace fa

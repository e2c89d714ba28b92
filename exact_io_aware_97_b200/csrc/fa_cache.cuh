// Writing new K and V rows into a paged cache held in e4m3 with one scale per block of
// `scale_block` tokens and head (sm_100a).
//
// For each (block, head) that receives rows: s = max(s_old, s_need), where s_need is the least
// power of two with max|x| <= 448 s over the new rows and s_old is the block's scale if it
// already holds rows of the sequence.  New rows are stored as e4m3(x / s); if s grew, the rows
// already there become e4m3(code * s_old / s).  With powers of two the division is exact and a
// rescaled code loses bits only below the smallest normal e4m3 value, so a block filled token by
// token ends as if filled at once, up to those bits.  A row that is not finite makes the scale
// of its block NaN.
//
// Bound by HBM for prompts (2 bytes read and 1 written per element; 67.6K rows of 8 heads, d = 128: 78
// us, 5.7 TB/s of the copy's 6.55) and by the chain of dependent loads (lengths, block table, scale,
// rows) for single tokens.  A unit is one (block, head): its warps hold the rows of K and V in
// registers (64 a thread, and 72 bytes of other values spilled), so a row is read once for the maximum
// and the rounding alike.
#pragma once

#include <cuda_fp16.h>

#include "fa_device.cuh"

namespace fa {

struct AppendParams {
  const __nv_bfloat16* src[2];  // k, v: [total, Hkv, D]
  uint8_t* pages[2];            // [num_pages, page_size, Hkv, D]
  float* scales[2];             // [num_pages, Hkv, page_size / scale_block]
  const int32_t* cu;            // [B + 1] or null: one row for each sequence
  const int32_t* block_table;
  const int32_t* seqlens;  // lengths with the new rows
  int B, total, Hkv, num_pages, page_shift, max_pages, sb_shift;
};

// Least power of two s with amax <= 448 s, at least 2^-126 (amax finite and > 0).
__device__ __forceinline__ float pow2_scale(float amax) {
  // 448 = 1.75 * 2^8; subnormal amax counts as an exponent of -126, below the floor anyway
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

// The sequence whose slots hold slot u: slots of sequence b start at (cu[b] >> sb_shift) + 2b,
// which leaves room for the at most (n_b >> sb_shift) + 2 blocks that n_b rows touch.
__device__ __forceinline__ int append_find(const int32_t* cu, int B, int sb_shift, int u) {
  int lo = 0, hi = B;  // slot start of lo is <= u; that of hi (if < B) is > u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((max(load_in(cu + mid), 0) >> sb_shift) + 2 * mid <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four codes of bf16 pairs w0, w1 times inv (a power of two: the bf16 product is exact wherever
// the code is not 0).
__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, __nv_bfloat162 inv) {
  const __nv_bfloat162 y0 = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w0), inv);
  const __nv_bfloat162 y1 = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w1), inv);
  return e4m3x4(__low2float(y0), __high2float(y0), __low2float(y1), __high2float(y1));
}

// The same divided by a scale that is no power of two (one that the cache had already), or NaN.
__device__ __noinline__ uint32_t quant4_div(uint32_t w0, uint32_t w1, float s) {
  return e4m3x4(__fdiv_rn(__uint_as_float(w0 << 16), s), __fdiv_rn(__uint_as_float(w0 & 0xFFFF0000u), s),
                __fdiv_rn(__uint_as_float(w1 << 16), s), __fdiv_rn(__uint_as_float(w1 & 0xFFFF0000u), s));
}

// Rows that a warp holds: 4 KB of K and V, 32 registers a lane, so that 32 warps fit an SM (16 rows
// for d = 128 too, with 16 warps per SM, took 84 us instead of 80 on the packed prompts).
template <int D>
constexpr int kAppendRows = 1024 / D;
constexpr int kAppendCta = 8;  // warps of a CTA

// Warps of a unit; one of more rows than a CTA holds is gone over twice (for scale blocks of 256 rows,
// d = 128: 95 us; 32 warps that hold it, one CTA per SM: 121 us).
template <int D>
__host__ __device__ __forceinline__ int append_warps(int sb_shift) {
  const int n = (1 << sb_shift) / kAppendRows<D>;
  return n < kAppendCta ? n : kAppendCta;
}

struct AppendUnit {
  int start, old, len;  // first new row of the sequence in the source; lengths before and after
  int blk0, page;       // first position of the block, its page
  int head, warp0;      // head of this warp; first warp of its unit
};

// One warp's rows of K and of V.  INSIDE: every row of the block is new.  The rows are loaded
// before the page (a load of its own, under way) and the scale are looked at.
template <int D, bool INSIDE>
__device__ __forceinline__ void append_rows(const AppendParams& p, const AppendUnit& t,
                                            uint32_t (&sm_max)[2][kAppendCta]) {
  constexpr int kLanes = D / 8;       // lanes of one row (8 values each)
  constexpr int kRows = 32 / kLanes;  // rows of one pass of a warp
  constexpr int kPass = kAppendRows<D> / kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpu = append_warps<D>(p.sb_shift), ps = 1 << p.page_shift;
  const int turns = (1 << p.sb_shift) / (wpu * kAppendRows<D>);  // of the unit's warps over its rows
  const bool alive = t.head < p.Hkv;
  int r0 = ((turns - 1) * wpu + warp - t.warp0) * kAppendRows<D> + lane / kLanes;  // first row, last turn
  const int col = (lane % kLanes) * 8;
  const long long pitch = (long long)p.Hkv * D;
  auto is_new = [&](int k) {
    const int pos = t.blk0 + r0 + k * kRows;
    return INSIDE || (pos >= t.old && pos < t.len);
  };

  uint4 x[2][kPass];
  auto load = [&] {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const __nv_bfloat16* src = p.src[w] + (t.start + t.blk0 + r0 - t.old) * pitch + t.head * D + col;
#pragma unroll
      for (int k = 0; k < kPass; ++k, src += kRows * pitch) {
        if (!INSIDE) x[w][k] = make_uint4(0u, 0u, 0u, 0u);
        if (alive && is_new(k)) x[w][k] = load_in(reinterpret_cast<const uint4*>(src));
      }
    }
  };
  // largest |x| as bits: the order of non-negative floats, infinity and NaN on top
  __nv_bfloat162 most[2] = {__float2bfloat162_rn(0.f), __float2bfloat162_rn(0.f)};
  auto look = [&] {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int k = 0; k < kPass; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          most[w] = __hmax2_nan(most[w], __habs2(reinterpret_cast<__nv_bfloat162*>(&x[w][k])[j]));
  };
  if (turns > 1) {
    const int step = wpu * kAppendRows<D>;
    r0 -= (turns - 1) * step;
#pragma unroll 1
    for (int i = 1; i < turns; ++i, r0 += step) {
      load();
      if (alive) look();
    }
  }
  load();
  if (t.page < 0 || t.page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrBadPage);
    return;
  }
  const int row_in_page = t.blk0 & (ps - 1);
  const long long at_scale =
      ((long long)t.page * p.Hkv + t.head) * (ps >> p.sb_shift) + (row_in_page >> p.sb_shift);
  float s_old[2] = {0.f, 0.f};
  if (!INSIDE && alive && t.blk0 < t.old) {
    s_old[0] = p.scales[0][at_scale];
    s_old[1] = p.scales[1][at_scale];
  }
  uint32_t top[2] = {0u, 0u};
  if (alive) {
    look();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t u = *reinterpret_cast<uint32_t*>(&most[w]);
      top[w] = __reduce_max_sync(0xffffffffu, max(u << 16, u & 0xFFFF0000u));
      if (wpu > 1 && lane == 0) sm_max[w][warp] = top[w];
    }
  }
  // a unit of several warps; and every warp has read the old scale before one writes the new one
  if (wpu > 1) __syncthreads();
  if (!alive) return;
  float s[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (wpu == kAppendCta)
      top[w] = __reduce_max_sync(0xffffffffu, sm_max[w][lane & (kAppendCta - 1)]);
    else if (wpu > 1)
      for (int k = 0; k < wpu; ++k) top[w] = max(top[w], sm_max[w][t.warp0 + k]);
    const float nan = __uint_as_float(0x7FC00000u);
    s[w] = top[w] >= 0x7F800000u ? nan : top[w] == 0u ? 0.f : pow2_scale(__uint_as_float(top[w]));
    if (!INSIDE) s[w] = (s[w] != s[w] || s_old[w] != s_old[w]) ? nan : fmaxf(s[w], s_old[w]);
  }
#pragma unroll 1
  for (int i = 0;;) {  // the last turn's rows are still here, the others are read again (from L2)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint8_t* const base = p.pages[w] + ((long long)t.page * ps + row_in_page + r0) * pitch + t.head * D + col;
      uint8_t* dst = base;
      const uint32_t bits = __float_as_uint(s[w]);
      if ((bits & 0x7FFFFFu) == 0u && bits <= 0x7E800000u) {  // 0 or a power of two up to 2^126
        // x / s is x * (1 / s): both round the same value once.  (Scale 0: all x are 0, and so are the
        // codes, without a sign.)
        const uint32_t up = (0x7F000000u - bits) >> 16, keep = bits ? 0xFFFFFFFFu : 0u;
        const uint32_t inv2 = up | up << 16;
        const __nv_bfloat162 inv = *reinterpret_cast<const __nv_bfloat162*>(&inv2);
#pragma unroll
        for (int k = 0; k < kPass; ++k, dst += kRows * pitch) {
          const uint4 v = x[w][k];
          if (is_new(k))
            *reinterpret_cast<uint2*>(dst) = make_uint2(quant4(v.x, v.y, inv) & keep, quant4(v.z, v.w, inv) & keep);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < kPass; ++k, dst += kRows * pitch) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int j = 0; j < kPass; ++j)
            if (j == k) v = x[w][j];
          if (is_new(k))
            *reinterpret_cast<uint2*>(dst) = make_uint2(quant4_div(v.x, v.y, s[w]), quant4_div(v.z, v.w, s[w]));
        }
      }
      if (!INSIDE && s[w] > s_old[w] && t.blk0 < t.old) {  // the scale grew: the rows held already move to it
        const float ratio = s_old[w] / s[w];
        dst = base;
#pragma unroll 1
        for (int k = 0; k < kPass && t.blk0 + r0 + k * kRows < t.old; ++k, dst += kRows * pitch) {
          uint2* to = reinterpret_cast<uint2*>(dst);
          const uint2 v = *to;
          uint32_t out[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t c = j ? v.y : v.x;
            out[j] = e4m3x4(e4m3_value(c & 255u) * ratio, e4m3_value((c >> 8) & 255u) * ratio,
                            e4m3_value((c >> 16) & 255u) * ratio, e4m3_value(c >> 24) * ratio);
          }
          *to = make_uint2(out[0], out[1]);
        }
      }
    }
    if (++i >= turns) break;
    r0 -= wpu * kAppendRows<D>;
    load();
  }
  if (wpu == 1) __syncwarp();  // every lane has read the old scales
  if (warp == t.warp0 && lane == 0) {
    p.scales[0][at_scale] = s[0];
    p.scales[1][at_scale] = s[1];
  }
}

// A CTA takes one block of rows for as many heads as its warps hold, K and V.
template <int D>
__global__ void __launch_bounds__(kAppendCta * 32, 4) fa_cache_append_kernel(const AppendParams p) {
  __shared__ uint32_t sm_max[2][kAppendCta];
  grid_wait();
  const int warp = threadIdx.x >> 5;
  const int wpu = append_warps<D>(p.sb_shift), upc = kAppendCta / wpu;  // warps of a unit, heads of a CTA

  if (p.cu && blockIdx.x == 0 && blockIdx.y == 0) {
    bool bad = threadIdx.x == 0 && (load_in(p.cu) < 0 || load_in(p.cu + p.B) > p.total);
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) bad |= load_in(p.cu + b) > load_in(p.cu + b + 1);
    if (bad) atomicOr(&g_error_word, kErrBadSeqlens);
  }
  const int u = blockIdx.x;
  const int b = p.cu ? append_find(p.cu, p.B, p.sb_shift, u) : u;
  const int start = p.cu ? load_in(p.cu + b) : b;
  const int end = p.cu ? load_in(p.cu + b + 1) : b + 1;
  const int idx = p.cu ? u - ((max(start, 0) >> p.sb_shift) + 2 * b) : 0;
  const int n = end - start, len = load_in(p.seqlens + b);
  // a slot before the first sequence's (rows before cu[0] belong to none), a sequence without new
  // rows, or one whose offsets or length cannot be used
  if (idx < 0 || start < 0 || end > p.total || n <= 0) return;
  if (n > len || (long long)len > (long long)p.max_pages << p.page_shift) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrBadSeqlens);
    return;
  }
  const int old = len - n;  // rows before the new ones
  AppendUnit t;
  t.start = start;
  t.old = old;
  t.len = len;
  t.blk0 = ((old >> p.sb_shift) + idx) << p.sb_shift;
  if (t.blk0 >= len) return;
  t.page = load_in(p.block_table + (long long)b * p.max_pages + (t.blk0 >> p.page_shift));
  t.head = blockIdx.y * upc + warp / wpu;
  t.warp0 = warp / wpu * wpu;
  if (t.blk0 >= old && t.blk0 + (1 << p.sb_shift) <= len)
    append_rows<D, true>(p, t, sm_max);
  else
    append_rows<D, false>(p, t, sm_max);
}

}  // namespace fa

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
// Bound by HBM for prompts (2 bytes read and 1 written per element) and by the chain of
// dependent loads (lengths, block table, scale, rows) for single tokens.  A unit is one
// (block, head) of K or of V: scale_block / 16 warps hold its rows in registers, 16 rows each,
// so a row is read once for the maximum and the rounding alike.
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
  return pack_e4m3x2_lo(a, b) | pack_e4m3x2_hi(c, d);
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
    if ((max(__ldg(cu + mid), 0) >> sb_shift) + 2 * mid <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Two e4m3 pairs of x / s, with x / s as x * inv where s is a power of two (the same value, since
// the product is exact up to its one rounding) and by division otherwise.
__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, float s, float inv, bool pow2) {
  float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u), __uint_as_float(w1 << 16),
                __uint_as_float(w1 & 0xFFFF0000u)};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = pow2 ? x[j] * inv : __fdiv_rn(x[j], s);
  return e4m3x4(x[0], x[1], x[2], x[3]);
}

// A CTA takes one block of rows for blockDim.x / 32 / (scale_block / 16) heads, K and V.  The rows
// are loaded as soon as the sequence is known, before the page and the scale.
template <int D>
__global__ void __launch_bounds__(512) fa_cache_append_kernel(const AppendParams p) {
  __shared__ uint32_t sm_max[2][16];
  constexpr int kLanes = D / 8;       // lanes of one row (8 values each)
  constexpr int kRows = 32 / kLanes;  // rows of one pass of a warp
  constexpr int kPass = 16 / kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpu = (1 << p.sb_shift) >> 4;   // warps of a unit
  const int upc = (blockDim.x >> 5) / wpu;  // heads of a CTA
  const int head = blockIdx.y * upc + warp / wpu;
  const int ps = 1 << p.page_shift;

  if (p.cu && blockIdx.x == 0 && blockIdx.y == 0) {
    bool bad = threadIdx.x == 0 && (__ldg(p.cu) < 0 || __ldg(p.cu + p.B) > p.total);
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) bad |= __ldg(p.cu + b) > __ldg(p.cu + b + 1);
    if (bad) atomicOr(&g_error_word, kErrBadSeqlens);
  }
  const int u = blockIdx.x;
  const int b = p.cu ? append_find(p.cu, p.B, p.sb_shift, u) : u;
  const int start = p.cu ? __ldg(p.cu + b) : b;
  const int end = p.cu ? __ldg(p.cu + b + 1) : b + 1;
  const int idx = p.cu ? u - ((max(start, 0) >> p.sb_shift) + 2 * b) : 0;
  const int n = end - start, len = __ldg(p.seqlens + b);
  // a sequence without new rows, or one whose offsets or length cannot be used
  if (start < 0 || end > p.total || n <= 0) return;
  if (n > len || (long long)len > (long long)p.max_pages << p.page_shift) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrBadSeqlens);
    return;
  }
  const int old = len - n;                                     // rows before the new ones
  const int blk0 = ((old >> p.sb_shift) + idx) << p.sb_shift;  // first position of the block
  if (blk0 >= len) return;
  const int page = __ldg(p.block_table + (long long)b * p.max_pages + (blk0 >> p.page_shift));
  const bool alive = head < p.Hkv;
  const int r0 = (warp % wpu) * 16 + lane / kLanes, col = (lane % kLanes) * 8;
  const long long pitch = (long long)p.Hkv * D;

  uint4 x[2][kPass];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const __nv_bfloat16* src = p.src[w] + (long long)(start + blk0 - old) * pitch + head * D + col;
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      const int r = r0 + k * kRows, pos = blk0 + r;
      x[w][k] = make_uint4(0u, 0u, 0u, 0u);
      if (alive && pos >= old && pos < len) x[w][k] = __ldcs(reinterpret_cast<const uint4*>(src + r * pitch));
    }
  }
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrBadPage);
    return;
  }
  const int row_in_page = blk0 & (ps - 1);
  const long long at_scale =
      ((long long)page * p.Hkv + head) * (ps >> p.sb_shift) + (row_in_page >> p.sb_shift);
  float s_old[2] = {0.f, 0.f};
  if (alive && blk0 < old) {
    s_old[0] = p.scales[0][at_scale];
    s_old[1] = p.scales[1][at_scale];
  }
  // largest |x| as bits: the order of non-negative floats, NaN and infinity on top
  uint32_t top[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t t2 = 0;
#pragma unroll
    for (int k = 0; k < kPass; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) t2 = __vmaxu2(t2, (&x[w][k].x)[j] & 0x7FFF7FFFu);
    top[w] = __reduce_max_sync(0xffffffffu, max(t2 << 16, t2 & 0xFFFF0000u));
    if (wpu > 1 && lane == 0) sm_max[w][warp] = top[w];
  }
  __syncthreads();  // (also: every warp has read the old scale before one writes the new one)
  if (!alive) return;
  const int first = warp / wpu * wpu;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (wpu > 1)
      for (int k = 0; k < wpu; ++k) top[w] = max(top[w], sm_max[w][first + k]);
    const float nan = __uint_as_float(0x7FC00000u);
    float s = top[w] >= 0x7F800000u ? nan : top[w] == 0u ? 0.f : pow2_scale(__uint_as_float(top[w]));
    s = (s != s || s_old[w] != s_old[w]) ? nan : fmaxf(s, s_old[w]);
    const float ratio = s > s_old[w] ? s_old[w] / s : 1.f, inv = __fdiv_rn(1.f, s);
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0u && s > 0.f;
    uint8_t* dst = p.pages[w] + ((long long)page * ps + row_in_page) * pitch + head * D + col;
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      const int r = r0 + k * kRows, pos = blk0 + r;
      uint2* to = reinterpret_cast<uint2*>(dst + r * pitch);
      if (pos >= old && pos < len) {
        const uint4 v = x[w][k];
        *to = s == 0.f ? make_uint2(0u, 0u)
                       : make_uint2(quant4(v.x, v.y, s, inv, pow2), quant4(v.z, v.w, s, inv, pow2));
      } else if (pos < old && ratio != 1.f) {
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
    if (warp == first && lane == 0) p.scales[w][at_scale] = s;
  }
}

}  // namespace fa

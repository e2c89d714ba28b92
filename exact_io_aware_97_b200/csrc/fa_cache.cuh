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

template <int D>
__global__ void __launch_bounds__(512) fa_cache_append_kernel(const AppendParams p) {
  __shared__ uint32_t sm_max[16];
  constexpr int kLanes = D / 8;           // lanes of one row (8 values each)
  constexpr int kRows = 32 / kLanes;      // rows of one pass of a warp
  constexpr int kPass = 16 / kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpu = (1 << p.sb_shift) >> 4;  // warps of a unit
  const int upc = (blockDim.x >> 5) / wpu;  // units (heads) of a CTA
  const int head = blockIdx.y * upc + warp / wpu;
  const int which = blockIdx.z;
  const int ps = 1 << p.page_shift;

  if (p.cu && blockIdx.x == 0 && blockIdx.y == 0 && which == 0) {
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
  const int old = len - n;                                    // rows before the new ones
  const int blk0 = ((old >> p.sb_shift) + idx) << p.sb_shift;  // first position of the block
  if (blk0 >= len) return;
  const int page = __ldg(p.block_table + (long long)b * p.max_pages + (blk0 >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrBadPage);
    return;
  }
  const bool alive = head < p.Hkv;
  const int row_in_page = blk0 & (ps - 1);
  float* scale = p.scales[which] + ((long long)page * p.Hkv + head) * (ps >> p.sb_shift) + (row_in_page >> p.sb_shift);
  const float s_old = (alive && blk0 < old) ? *scale : 0.f;
  const int r0 = (warp % wpu) * 16 + lane / kLanes, col = (lane % kLanes) * 8;
  const __nv_bfloat16* src = p.src[which] + ((long long)(start + blk0 - old) * p.Hkv + head) * D + col;
  uint8_t* dst = p.pages[which] + (((long long)page * ps + row_in_page) * p.Hkv + head) * D + col;

  uint4 x[kPass];
  uint32_t top = 0;  // largest |x| as bits: the order of non-negative floats, NaN and inf on top
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int r = r0 + k * kRows, pos = blk0 + r;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (alive && pos >= old && pos < len)
      x[k] = *reinterpret_cast<const uint4*>(src + (long long)r * p.Hkv * D);
  }
#pragma unroll
  for (int k = 0; k < kPass; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = (&x[k].x)[j];
      top = max(top, max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
    }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) sm_max[warp] = top;
  __syncthreads();
  for (int w = warp / wpu * wpu; w < (warp / wpu + 1) * wpu; ++w) top = max(top, sm_max[w]);
  if (!alive) return;
  const float nan = __uint_as_float(0x7FC00000u);
  float s = top >= 0x7F800000u ? nan : top == 0u ? 0.f : pow2_scale(__uint_as_float(top));
  s = (s != s || s_old != s_old) ? nan : fmaxf(s, s_old);
  const float ratio = s > s_old ? s_old / s : 1.f;
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int r = r0 + k * kRows, pos = blk0 + r;
    uint8_t* to = dst + (long long)r * p.Hkv * D;
    if (pos >= old && pos < len) {
      uint32_t out[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w0 = (&x[k].x)[2 * j], w1 = (&x[k].x)[2 * j + 1];
        const float a = __uint_as_float(w0 << 16), bq = __uint_as_float(w0 & 0xFFFF0000u);
        const float c = __uint_as_float(w1 << 16), dq = __uint_as_float(w1 & 0xFFFF0000u);
        out[j] = s == 0.f ? 0u : e4m3x4(__fdiv_rn(a, s), __fdiv_rn(bq, s), __fdiv_rn(c, s), __fdiv_rn(dq, s));
      }
      *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
    } else if (pos < old && ratio != 1.f) {
      const uint2 w = *reinterpret_cast<const uint2*>(to);
      uint32_t out[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t v = j ? w.y : w.x;
        out[j] = e4m3x4(e4m3_value(v & 255u) * ratio, e4m3_value((v >> 8) & 255u) * ratio,
                        e4m3_value((v >> 16) & 255u) * ratio, e4m3_value(v >> 24) * ratio);
      }
      *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
    }
  }
  if (warp % wpu == 0 && lane == 0) *scale = s;
}

}  // namespace fa

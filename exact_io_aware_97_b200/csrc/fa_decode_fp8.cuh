// Decode attention over a paged cache held in e4m3 with a scale for each block of tokens and
// head (sm_100a).
//
// Query token i (of Nq new tokens) and query head h of a sequence of `len` tokens (the new ones
// included) attend to cache rows j <= len - Nq + i of K/V head h / G:
//   t_j = scale * sk_j * (q . k_j),  p_j = e^(t_j - m),  o = sum_j p_j sv_j v_j / sum_j p_j,
// where k_j, v_j are the stored e4m3 values and sk_j, sv_j the scales of their blocks.
//
// One CTA takes one (sequence, query token, query head): its four warps walk the rows with a
// running maximum and sum each and merge in shared memory.
#pragma once

#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "fa_device.cuh"

namespace fa {

struct Dec8Params {
  const __nv_bfloat16* q;  // [B, Nq, Hq, D]
  const uint8_t* pages[2];
  const float* scales[2];  // [num_pages, Hkv, page_size >> sb_shift]
  const int32_t* block_table;
  const int32_t* seqlens;
  __nv_bfloat16* o;
  float* lse;  // [B, Hq, Nq] or null
  int B, Nq, Hq, Hkv, G, num_pages, page_shift, sb_shift, max_pages;
  float tau;  // scale * log2(e)
};

template <int D>
__global__ void __launch_bounds__(128) fa_decode_fp8_kernel(const Dec8Params p) {
  constexpr int V = D / 32;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, kvh = h / p.G;
  const long long cap = (long long)p.max_pages << p.page_shift;
  const int len = (int)min((long long)max(__ldg(p.seqlens + b), 0), cap);
  const int n = len - p.Nq + 1 + i;  // rows this query sees (may be <= 0)
  const long long qrow = ((long long)b * p.Nq + i) * p.Hq + h;
  float q[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    q[v] = __bfloat162float(p.q[qrow * D + lane * V + v]);
    acc[v] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int psm = (1 << p.page_shift) - 1, nb_shift = p.page_shift - p.sb_shift;
  for (int j = warp; j < n; j += 4) {
    int page = __ldg(p.block_table + (long long)b * p.max_pages + (j >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
      atomicOr(&g_error_word, kErrBadPage);
      page = 0;
    }
    const int r = j & psm;
    const long long at = ((((long long)page << p.page_shift) + r) * p.Hkv + kvh) * D + lane * V;
    const long long sat = (((long long)page * p.Hkv + kvh) << nb_shift) + (r >> p.sb_shift);
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s = fmaf(q[v], e4m3_value(p.pages[0][at + v]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float t = s * (p.scales[0][sat] * p.tau);
    const float m_new = fmaxf(m, t);
    const float alpha = (m_new == -INFINITY) ? 1.f : exp2f(m - m_new);
    const float pj = exp2f(t - ((m_new == -INFINITY) ? 0.f : m_new));
    l = l * alpha + pj;
    const float w = pj * p.scales[1][sat];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, e4m3_value(p.pages[1][at + v]), acc[v] * alpha);
    m = m_new;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sm_o[warp][lane * V + v] = acc[v];
  __syncthreads();
  if (warp != 0) return;
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w]);
  float a[V];
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float e = (M == -INFINITY) ? (sm_l[w] == 0.f ? 0.f : 1.f) : exp2f(sm_m[w] - M);
    L += e * sm_l[w];
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] += e * sm_o[w][lane * V + v];
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that sees nothing: o = 0, lse = -inf
#pragma unroll
  for (int v = 0; v < V; ++v) p.o[qrow * D + lane * V + v] = __float2bfloat16_rn(a[v] * inv);
  if (lane == 0 && p.lse)
    p.lse[((long long)b * p.Hq + h) * p.Nq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace fa

// Rotary positions for q and k (sm_100a).
//
// Column pair i of a head turns by the angle pos * w_i:
//   y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin),
// where (a, b) = (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved") for i < rot/2 and the
// columns from rot on are copied.  The gradient of x is the same with -sin, so one kernel does
// both directions.
//
// The angle is reduced in fp64 as a fraction of a turn (pos * w / 2 pi minus its nearest
// integer), so a position of millions loses nothing; sine and cosine of the reduced angle, and
// the products, are fp32, rounded once on output.
//
// Bound by HBM: every element is read and written once.  One warp owns one (token, run of
// heads): its lanes hold the sines and cosines of their own columns in registers for all heads
// of the run, so no shared memory, barrier or table in device memory is involved.
#pragma once

#include "fa_device.cuh"

namespace fa {

struct RopeParams {
  const void* x[2];  // q, k (k may have no heads)
  void* y[2];
  long long xs[2], ys[2];  // elements from one token to the next
  int heads[2];
  const int32_t* positions;  // [rows] or null: row % period
  const double* freqs;       // [rot / 2], radians per position
  long long rows;
  int period, rot, interleaved, backward;
  float amplitude;
  int chunks, per_chunk;  // the heads of a token are cut into `chunks` runs of `per_chunk`
};

// cos and sin of pair i at a position, times the amplitude
__device__ __forceinline__ float2 rope_cs(const RopeParams& p, int i, double pos) {
  const double t = pos * __ldg(p.freqs + i) * 0.15915494309189533577;  // turns
  float s, c;
  sincospif((float)(2.0 * (t - rint(t))), &s, &c);
  s *= p.amplitude;
  return make_float2(c * p.amplitude, p.backward ? -s : s);
}

__device__ __forceinline__ double rope_pos(const RopeParams& p, long long row) {
  return p.positions ? (double)__ldg(p.positions + row) : (double)(row % p.period);
}

__device__ __forceinline__ float rope_load(const float* x) { return *x; }
__device__ __forceinline__ float rope_load(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ void rope_store(float* y, float v) { *y = v; }
__device__ __forceinline__ void rope_store(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

// Any even rot: one lane per pair of columns (or per copied column).
template <typename T, int D>
__global__ void __launch_bounds__(256) fa_rope_kernel(const RopeParams p) {
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long row = unit / p.chunks;
  if (row >= p.rows) return;
  const int h0 = (int)(unit - row * p.chunks) * p.per_chunk;
  const int h1 = min(h0 + p.per_chunk, p.heads[0] + p.heads[1]);
  const double pos = rope_pos(p, row);
  const int np = p.rot / 2, nitem = np + D - p.rot;
  for (int i = lane; i < nitem; i += 32) {
    const bool turn = i < np;
    const float2 cs = turn ? rope_cs(p, i, pos) : make_float2(1.f, 0.f);
    const int a = !turn ? p.rot + i - np : p.interleaved ? 2 * i : i;
    const int b = p.interleaved ? a + 1 : a + np;
    for (int h = h0; h < h1; ++h) {
      const int w = h >= p.heads[0];
      const int hh = w ? h - p.heads[0] : h;
      const T* x = static_cast<const T*>(p.x[w]) + row * p.xs[w] + (long long)hh * D;
      T* y = static_cast<T*>(p.y[w]) + row * p.ys[w] + (long long)hh * D;
      if (turn) {
        const float u = rope_load(x + a), v = rope_load(x + b);
        rope_store(y + a, fmaf(u, cs.x, -v * cs.y));
        rope_store(y + b, fmaf(v, cs.x, u * cs.y));
      } else {
        y[a] = x[a];
      }
    }
  }
}

}  // namespace fa

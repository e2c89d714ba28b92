// Rotary positions for q and k (sm_100a).
//
// Column pair i of a head turns by the angle pos * w_i:
//   y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin),
// where (a, b) = (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved") for i < rot/2 and the
// columns from rot on are copied.  The gradient of x is the same with -sin, so one kernel does
// both directions.
//
// The angle is reduced in fp64 as a fraction of a turn (pos * w / 2 pi minus its nearest
// integer), so a position of millions loses nothing; sine and cosine of the reduced angle are fp32, with
// what its own rounding to fp32 took put back to first order, and the products are fp32, rounded once on
// output.
//
// Bound by HBM: every element is read and written once (8192 rows of 72 heads, d = 128, bf16: 50.5 us, 6.0
// TB/s of the 6.55 that a copy reaches; 32749 rows of 40 heads: 106 us, 6.3 TB/s).  One warp owns one (token, run of
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
  const double t = pos * load_in(p.freqs + i) * 0.15915494309189533577;  // turns
  const double half = 2.0 * (t - rint(t));  // half turns
  const float near = (float)half, off = (float)(half - near) * 3.14159265f;
  float s, c;
  sincospif(near, &s, &c);
  const float s0 = s;
  s = fmaf(c, off, s);  // what the rounding of the angle took (its square is far below fp32)
  c = fmaf(-s0, off, c);
  s *= p.amplitude;
  return make_float2(c * p.amplitude, p.backward ? -s : s);
}

__device__ __forceinline__ double rope_pos(const RopeParams& p, long long row) {
  return p.positions ? (double)load_in(p.positions + row) : (double)(row % p.period);
}

__device__ __forceinline__ float rope_load(const float* x) { return *x; }
__device__ __forceinline__ float rope_load(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ void rope_store(float* y, float v) { *y = v; }
__device__ __forceinline__ void rope_store(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

// Any even rot in the half layout: one lane per pair of columns (or per copied column); what the
// vectors below cannot take (8192 rows as above: 184 us for rot = 128 in this way, 315 for 120, 92 or 74).
template <typename T, int D>
__global__ void __launch_bounds__(256) fa_rope_kernel(const RopeParams p) {
  grid_wait();
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
    const int a = turn ? i : p.rot + i - np, b = a + np;
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

// Rows in 16-byte vectors.  A lane owns one slot of a head, two vectors: columns that turn
// together (half layout), neighbours (interleaved), or neighbours that are copied.  The lanes of
// a warp cover 32 / slots heads at a time; each computes a share of its slot's sines and cosines
// and gets the rest from the lanes of the same slot.  Half layout: rot / 2 is a multiple of the
// vector (else fa_rope_kernel).
template <typename T>
struct RopeVec;
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = (&w.x)[j];
      x[2 * j] = __uint_as_float(u << 16);
      x[2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct RopeVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float((&w.x)[j]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256) fa_rope_vec_kernel(const RopeParams p) {
  using X = RopeVec<T>;
  constexpr int V = X::N, kSlots = D / (2 * V), kHeads = 32 / kSlots, kShare = V / kHeads, kUnroll = 4;
  grid_wait();
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, slot = lane % kSlots, sub = lane / kSlots;
  const long long row = unit / p.chunks;
  if (row >= p.rows) return;
  const int h0 = (int)(unit - row * p.chunks) * p.per_chunk;
  const int nh = p.heads[0] + p.heads[1], h1 = min(h0 + p.per_chunk, nh);
  const int np = p.rot / 2;
  const double pos = rope_pos(p, row);
  float2 own[kShare];
#pragma unroll
  for (int j = 0; j < kShare; ++j) {
    const int i = slot * V + sub * kShare + j;
    own[j] = i < np ? rope_cs(p, i, pos) : make_float2(1.f, 0.f);
  }
  float c[V], s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int from = (j / kShare) * kSlots + slot;
    c[j] = __shfl_sync(0xffffffffu, own[j % kShare].x, from);
    s[j] = __shfl_sync(0xffffffffu, own[j % kShare].y, from);
  }
  const int pairs = min(max(np - slot * V, 0), V);  // of this slot that turn
  int ca, cb;                                       // first columns of the two vectors
  if (INTER) {
    ca = slot * 2 * V;
    cb = ca + V;
  } else {
    ca = pairs ? slot * V : p.rot + (slot - np / V) * 2 * V;
    cb = pairs ? ca + np : ca + V;
  }
  const T* const xq = static_cast<const T*>(p.x[0]) + row * p.xs[0];
  const T* const xk = static_cast<const T*>(p.x[1]) + row * p.xs[1] - (long long)p.heads[0] * D;
  T* const yq = static_cast<T*>(p.y[0]) + row * p.ys[0];
  T* const yk = static_cast<T*>(p.y[1]) + row * p.ys[1] - (long long)p.heads[0] * D;
  for (int h = h0 + sub; h < h1; h += kHeads * kUnroll) {
    uint4 wa[kUnroll], wb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u * kHeads;
      if (hh < h1) {
        const T* x = (hh < p.heads[0] ? xq : xk) + (long long)hh * D;
        wa[u] = *reinterpret_cast<const uint4*>(x + ca);
        wb[u] = *reinterpret_cast<const uint4*>(x + cb);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u * kHeads;
      if (hh >= h1) continue;
      if (pairs) {
        float a[V], b[V];
        X::unpack(wa[u], a);
        X::unpack(wb[u], b);
        if (INTER) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float& x0 = 2 * j < V ? a[(2 * j) % V] : b[(2 * j) % V];
            float& x1 = 2 * j < V ? a[(2 * j + 1) % V] : b[(2 * j + 1) % V];
            const float y0 = fmaf(x0, c[j], -x1 * s[j]), y1 = fmaf(x1, c[j], x0 * s[j]);
            x0 = j < pairs ? y0 : x0;
            x1 = j < pairs ? y1 : x1;
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float x0 = a[j], x1 = b[j];
            a[j] = fmaf(x0, c[j], -x1 * s[j]);
            b[j] = fmaf(x1, c[j], x0 * s[j]);
          }
        }
        wa[u] = X::pack(a);
        wb[u] = X::pack(b);
      }
      T* y = (hh < p.heads[0] ? yq : yk) + (long long)hh * D;
      *reinterpret_cast<uint4*>(y + ca) = wa[u];
      *reinterpret_cast<uint4*>(y + cb) = wb[u];
    }
  }
}

}  // namespace fa

// Host side of the C ABI declared in include/fa.h: argument checks, TMA descriptors,
// workspace carving and kernel launches.  No device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/fa.h"
#include "fa_bwd_sm100.cuh"
#include "fa_cache.cuh"
#include "fa_decode_fp8.cuh"
#include "fa_decode_fp8_narrow.cuh"
#include "fa_decode_fp8_tc.cuh"
#include "fa_decode_sm100.cuh"
#include "fa_fwd_sm100.cuh"
#include "fa_pages.cuh"
#include "fa_rope.cuh"

namespace fa {

// fp32 -> bf16 (round to nearest even), used when the forward is called with fp32 inputs.
__global__ void cast_f32_bf16_kernel(const float* __restrict__ src, __nv_bfloat16* __restrict__ dst, size_t n) {
  const size_t n4 = n / 4;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += stride) {
    const float4 x = reinterpret_cast<const float4*>(src)[i];
    uint2 w;
    w.x = pack_bf16x2(x.x, x.y);
    w.y = pack_bf16x2(x.z, x.w);
    reinterpret_cast<uint2*>(dst)[i] = w;
  }
  for (size_t i = n4 * 4 + (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride)
    dst[i] = __float2bfloat16_rn(src[i]);
}

// V^T for the fp8 forward: vt[(b*Hkv + h)*128 + c][n] = v[b][n][h][c] for n < Nk, 0 up to
// NkPad (so that padded keys hold finite values; they are masked).  One block per (64-key
// chunk, head, sequence), staged through shared memory so both sides are coalesced.
__global__ void __launch_bounds__(256) transpose_v_e4m3_kernel(const uint8_t* __restrict__ v, uint8_t* __restrict__ vt,
                                                               int Nk, int Hkv, int NkPad) {
  __shared__ uint32_t tile[64][33];  // 64 keys x 128 bytes (32 words), padded
  const int n0 = blockIdx.x * 64, h = blockIdx.y, b = blockIdx.z;
  for (int idx = threadIdx.x; idx < 64 * 32; idx += 256) {
    const int r = idx >> 5, w = idx & 31;
    const int n = n0 + r;
    tile[r][w] = (n < Nk) ? reinterpret_cast<const uint32_t*>(v + (((size_t)b * Nk + n) * Hkv + h) * 128)[w] : 0u;
  }
  __syncthreads();
  // each thread writes 4 consecutive keys (one word) of one column c
  for (int idx = threadIdx.x; idx < 128 * 16; idx += 256) {
    const int c = idx >> 4, kq = idx & 15;  // column, group of four keys
    const int n = n0 + 4 * kq;
    if (n >= NkPad) continue;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) word |= ((tile[4 * kq + e][c >> 2] >> (8 * (c & 3))) & 0xFFu) << (8 * e);
    *reinterpret_cast<uint32_t*>(vt + (((size_t)b * Hkv + h) * 128 + c) * NkPad + n) = word;
  }
}

// fp32 -> the nearest tf32 value (10 mantissa bits, ties to even), kept in fp32 storage.
// Integer rounding on the bit pattern; infinities and NaN pass through.
__device__ __forceinline__ float round_tf32(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7F800000u) != 0x7F800000u) {
    u += 0x0FFFu + ((u >> 13) & 1u);
    u &= ~0x1FFFu;
  }
  return __uint_as_float(u);
}

__global__ void round_tf32_kernel(const float* __restrict__ src, float* __restrict__ dst, size_t n) {
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) dst[i] = round_tf32(src[i]);
}

// V^T for the tf32 forward (d = 64, fp32, rounded to tf32): vt[(b*Hkv + h)*64 + c][n] =
// v[b][n][h][c] for n < Nk, 0 up to NkPad.  One block per (32-key chunk, head, sequence).
__global__ void __launch_bounds__(256) transpose_v_f32_kernel(const float* __restrict__ v, float* __restrict__ vt,
                                                              int Nk, int Hkv, int NkPad) {
  __shared__ float tile[32][65];
  const int n0 = blockIdx.x * 32, h = blockIdx.y, b = blockIdx.z;
  for (int idx = threadIdx.x; idx < 32 * 64; idx += 256) {
    const int r = idx >> 6, c = idx & 63;
    const int n = n0 + r;
    tile[r][c] = (n < Nk) ? round_tf32(v[(((size_t)b * Nk + n) * Hkv + h) * 64 + c]) : 0.f;
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < 64 * 32; idx += 256) {
    const int c = idx >> 5, r = idx & 31;
    const int n = n0 + r;
    if (n < NkPad) vt[(((size_t)b * Hkv + h) * 64 + c) * NkPad + n] = tile[r][c];
  }
}

// Reads and clears the error word in one atomic step, so that a record made by a kernel on
// another stream between a read and a separate clear cannot be lost.
__global__ void take_error_word_kernel() { g_error_taken = atomicExch(&g_error_word, 0u); }

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// [rows, heads, D] bf16 tensor (D innermost) seen as a 3-D map {D, heads, rows}; box of
// 64 columns x 1 head x box_rows rows with the 128-byte swizzle.  Consecutive rows are
// row_stride elements apart (heads * D when the tensor is dense; 3 * heads * D for one of
// q, k, v inside a packed [rows, 3, heads, D] tensor).
bool make_map(CUtensorMap* map, const void* base, int D, int heads, int64_t rows, int box_rows,
              int64_t row_stride = 0) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  if (row_stride <= 0) row_stride = (int64_t)heads * D;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)row_stride * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Byte tensor (e4m3 stored as bytes) of three dimensions with the 128-byte swizzle.
bool make_map_u8(CUtensorMap* map, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                 const cuuint32_t (&box)[3]) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 tensor of three dimensions with the 128-byte swizzle (box inner extent 32 elements).
bool make_map_f32(CUtensorMap* map, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                  const cuuint32_t (&box)[3]) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Dense bf16 output [rows, heads, D] as the TMA store target of the forward epilogue: box of
// 16 columns x 1 head x 32 rows (one softmax warp's rows) with the 32-byte swizzle.
bool make_map_o(CUtensorMap* map, const void* base, int D, int heads, int64_t rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc || rows <= 0 || (reinterpret_cast<uintptr_t>(base) & 15u) != 0) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
  cuuint32_t box[3] = {16, 1, 32};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Work units of the forward: 256 query rows of one head, or, at fixed length when the query
// heads of every K/V group come in pairs, 128 rows of two heads of one group: both tiles of a
// unit then see the same keys, so a causal unit has no step with one tile (8K GQA causal:
// 1259 -> 1286 TFLOP/s, FP8 1415 -> 1473, same box).  Packed varlen inputs keep 256-row
// units (measured 1124 against 1114 TFLOP/s with pairs on the 16-sequence workload; the
// kernel supports both).  Sets prm.hpair and prm.T; returns the number of units (fixed
// length) or 0 (varlen: counted on the device).
int64_t fwd_units(FwdParams& prm, bool varlen, int64_t rows_q) {
  (void)rows_q;
  prm.hpair = (prm.G % 2 == 0 && !varlen) ? 1 : 0;
  const int ur = kUnitRows >> prm.hpair;
  prm.T = varlen ? 0 : (prm.Nq + ur - 1) / ur;
  return varlen ? 0 : (int64_t)prm.T * prm.B * (prm.Hq >> prm.hpair);
}

int sm_count_cached() {
  static int counts[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (counts[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    counts[dev] = n;
  }
  return counts[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

template <class K>
cudaError_t set_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// A launch whose blocks may come while the stream's last kernel ends; the kernel waits for its results
// (grid_wait) before it touches memory.  (1 to 2 us less between kernels, and 0.5 us less on the host.)
template <class... P, class... A>
bool launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return true;
  (void)cudaGetLastError();  // reported here, not by a later call
  return false;
}

// set_smem, once for each device (a call on this path is a few microseconds altogether).
template <class K>
bool set_smem_once(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (done.load(std::memory_order_relaxed) >> dev & 1u) return true;
  if (set_smem(kernel, bytes) != cudaSuccess) return false;
  done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return true;
}

template <int D, bool F32>
fa_status launch_fwd(const void* q, const void* k, const void* v, const FwdParams& prm, int64_t rows_q,
                     int64_t rows_k, int units, cudaStream_t st, int64_t q_stride = 0, int64_t kv_stride = 0) {
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q, D, prm.Hq, rows_q, kBM, q_stride) || !make_map(&mk, k, D, prm.Hkv, rows_k, kBN, kv_stride) ||
      !make_map(&mv, v, D, prm.Hkv, rows_k, kBN, kv_stride))
    return FA_ERR_CUDA;
  // bf16 O goes out through TMA stores when it can be described (16-byte aligned base); the
  // kernel writes per lane otherwise (and always for fp32 O)
  FwdParams p2 = prm;
  CUtensorMap mo = mq;
  p2.o_tma = (!F32 && make_map_o(&mo, prm.o, D, prm.Hq, rows_q)) ? 1 : 0;
  auto kern = fa_fwd_kernel<D, F32>;
  const int smem = FwdCfg<D>::kSmemBytes;
  if (set_smem(kern, smem) != cudaSuccess) return FA_ERR_CUDA;
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  const int grid = (units > 0) ? std::min(units, sms) : sms;
  kern<<<grid, kFwdThreads, smem, st>>>(mq, mk, mv, mo, p2);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
fa_status launch_decode(const void* kc, const void* vc, const DecParams& prm, cudaStream_t st) {
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)prm.B * prm.Lmax;
  if (!make_map(&mk, kc, D, prm.Hkv, rows, kDecKeys) || !make_map(&mv, vc, D, prm.Hkv, rows, kDecKeys))
    return FA_ERR_CUDA;
  auto ks = fa_decode_split_kernel<D, false>;
  const int smem = DecCfg<D>::kSmemBytes;
  if (set_smem(ks, smem) != cudaSuccess) return FA_ERR_CUDA;
  dim3 grid(prm.nsplit, prm.Hkv, prm.B);
  ks<<<grid, kDecThreads, smem, st>>>(mk, mv, prm);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  const int nbh = prm.B * prm.Hq;
  fa_decode_combine_kernel<D><<<(nbh + 3) / 4, 128, 0, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
fa_status launch_decode_paged(const void* kp, const void* vp, const DecParams& prm, cudaStream_t st) {
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)prm.num_pages << prm.page_shift;
  if (!make_map(&mk, kp, D, prm.Hkv, rows, prm.page_box) || !make_map(&mv, vp, D, prm.Hkv, rows, prm.page_box))
    return FA_ERR_CUDA;
  auto ks = fa_decode_split_kernel<D, true>;
  const int smem = DecCfg<D>::kSmemBytes;
  if (set_smem(ks, smem) != cudaSuccess) return FA_ERR_CUDA;
  dim3 grid(prm.nsplit, prm.Hkv, prm.B);
  ks<<<grid, kDecThreads, smem, st>>>(mk, mv, prm);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  const int nbh = prm.B * prm.Hq;
  fa_decode_combine_kernel<D><<<(nbh + 3) / 4, 128, 0, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Fixed length (prm.cu null) or packed varlen rows (prm.cu, prm.total, prm.ntiles set).
template <int D>
fa_status launch_bwd(const void* q, const void* k, const void* v, const BwdParams& prm, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mdo;
  const bool varlen = prm.cu != nullptr;
  const int64_t rows_q = varlen ? (int64_t)prm.total : (int64_t)prm.B * prm.Nq;
  const int64_t rows_k = varlen ? (int64_t)prm.total : (int64_t)prm.B * prm.Nk;
  if (!make_map(&mq, q, D, prm.Hq, rows_q, kBwdTile) || !make_map(&mdo, prm.dout, D, prm.Hq, rows_q, kBwdTile) ||
      !make_map(&mk, k, D, prm.Hkv, rows_k, kBwdTile) || !make_map(&mv, v, D, prm.Hkv, rows_k, kBwdTile))
    return FA_ERR_CUDA;
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  if (varlen) fa_bwd_tiles_kernel<<<1, kTilesThreads, 0, st>>>(prm);
  const long long pre_rows =
      varlen ? (long long)prm.Hq * prm.ntiles * kBwdTile : (long long)prm.B * prm.Hq * prm.NqPad;
  const int pre_blocks = (int)std::min<long long>((pre_rows + 7) / 8, (long long)sms * 16);
  if (pre_blocks > 0) fa_bwd_pre_kernel<D><<<pre_blocks, 256, 0, st>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (rows_k > 0 && (varlen || prm.Nk > 0)) {
    // one CTA per (key tile, K/V head, sequence), tile-major (the kernels' bwd_cta_coords);
    // varlen: a tile number over all sequences (bounded by ntiles; the kernels find the
    // sequence and leave numbers past the last tile idle)
    const long long ctas = varlen ? (long long)prm.ntiles * prm.Hkv
                                  : (long long)((prm.Nk + kBwdTile - 1) / kBwdTile) * prm.Hkv * prm.B;
    if (ctas >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ctas);
    if (D == 128) {
      // pairs of 64 queries, two in flight: Q and dO maps with 64-row boxes
      CUtensorMap mq64, mdo64;
      if (!make_map(&mq64, q, D, prm.Hq, rows_q, kBwdQ) || !make_map(&mdo64, prm.dout, D, prm.Hq, rows_q, kBwdQ))
        return FA_ERR_CUDA;
      // the fp32 dQ accumulator as a TMA reduce target: {d, Hq, rows}, box 128 x 1 x 64, no swizzle
      CUtensorMap mdq;
      const cuuint64_t ddq[3] = {(cuuint64_t)D, (cuuint64_t)prm.Hq, (cuuint64_t)rows_q};
      const cuuint64_t sdq[2] = {(cuuint64_t)D * 4, (cuuint64_t)prm.Hq * D * 4};
      const cuuint32_t bdq[3] = {(cuuint32_t)D, 1, (cuuint32_t)kBwdQ};
      const cuuint32_t edq[3] = {1, 1, 1};
      EncodeTiledFn enc = get_encode_fn();
      if (!enc || enc(&mdq, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, prm.dq_acc, ddq, sdq, bdq, edq,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return FA_ERR_CUDA;
      const int smem = Bwd2Cfg::kSmemBytes;
      if (set_smem(fa_bwd2_kernel, smem) != cudaSuccess) return FA_ERR_CUDA;
      fa_bwd2_kernel<<<grid, kBwdThreads, smem, st>>>(mq64, mk, mv, mdo64, mdq, prm);
    } else {
      auto kern = fa_bwd_kernel<D>;
      const int smem = BwdCfg<D>::kSmemBytes;
      if (set_smem(kern, smem) != cudaSuccess) return FA_ERR_CUDA;
      kern<<<grid, kBwdThreads, smem, st>>>(mq, mk, mv, mdo, prm);
    }
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  const size_t n4 = (size_t)rows_q * prm.Hq * D / 4;
  if (n4 > 0) fa_bwd_dq_kernel<D><<<(int)std::min<size_t>((n4 + 255) / 256, (size_t)sms * 8), 256, 0, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

int fa_device_sm_count(void) { return sm_count_cached(); }

size_t fa_fwd_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d, fa_dtype in_dtype, int varlen) {
  if (in_dtype == FA_TF32) {
    // tf32-rounded copies of q and k, then the rounded, transposed v
    if (varlen || B <= 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nk < 0 || d != 64) return 0;
    const size_t pad = (size_t)(Nk + 3) / 4 * 4;
    return align_up((size_t)B * Nq * Hq * d * 4, 256) + align_up((size_t)B * Nk * Hkv * d * 4, 256) +
           align_up((size_t)B * Hkv * d * pad * 4, 256);
  }
  if (in_dtype != FA_F32) return 0;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nk < 0 || d <= 0) return 0;
  // bf16 copies of q, k, v (varlen: Nq = Nk = the packed row count)
  const size_t rq = varlen ? (size_t)Nq : (size_t)B * Nq, rk = varlen ? (size_t)Nk : (size_t)B * Nk;
  const size_t nq = rq * Hq * d, nk = rk * Hkv * d;
  return align_up(nq * 2, 256) + 2 * align_up(nk * 2, 256);
}

}  // extern "C"

namespace fa {
namespace {

// fp32 q, k, v (d = 64, fixed length) on the tf32 tensor-core path; O written as fp32.
fa_status fwd_tf32(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                   int Nk, float scale, int causal, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  constexpr int D = 64;
  const int64_t rows_q = (int64_t)B * Nq, rows_k = (int64_t)B * Nk;
  const int pad = (Nk + 3) / 4 * 4;
  const size_t need = fa_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, D, FA_TF32, 0);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return FA_ERR_WORKSPACE;
  if (B > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t nq = (size_t)rows_q * Hq * D, nk = (size_t)rows_k * Hkv * D;
  float* qr = reinterpret_cast<float*>(ws);
  float* kr = reinterpret_cast<float*>(ws + align_up(nq * 4, 256));
  float* vt = reinterpret_cast<float*>(ws + align_up(nq * 4, 256) + align_up(nk * 4, 256));
  const int sms0 = std::max(sm_count_cached(), 1);
  round_tf32_kernel<<<sms0 * 4, 256, 0, st>>>(static_cast<const float*>(q), qr, nq);
  if (Nk > 0) {
    round_tf32_kernel<<<sms0 * 4, 256, 0, st>>>(static_cast<const float*>(k), kr, nk);
    dim3 g((pad + 31) / 32, Hkv, B);
    transpose_v_f32_kernel<<<g, 256, 0, st>>>(static_cast<const float*>(v), vt, Nk, Hkv, pad);
  }
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  FwdParams prm{};
  prm.o = o;
  prm.lse = lse;
  prm.cu = nullptr;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Nq = Nq;
  prm.Nk = Nk;
  prm.causal = causal ? 1 : 0;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  prm.o_scale = 1.f;
  const int64_t units64 = fwd_units(prm, false, rows_q);
  if (units64 >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  const cuuint64_t dq3[3] = {D, (cuuint64_t)Hq, (cuuint64_t)rows_q};
  const cuuint64_t sq2[2] = {D * 4, (cuuint64_t)Hq * D * 4};
  const cuuint64_t dk3[3] = {D, (cuuint64_t)Hkv, (cuuint64_t)std::max<int64_t>(rows_k, 1)};
  const cuuint64_t sk2[2] = {D * 4, (cuuint64_t)Hkv * D * 4};
  const int vp = std::max(pad, 4);
  const cuuint64_t dv3[3] = {(cuuint64_t)vp, D, (cuuint64_t)B * Hkv};
  const cuuint64_t sv2[2] = {(cuuint64_t)vp * 4, (cuuint64_t)vp * 4 * D};
  const cuuint32_t box_rows[3] = {32, 1, (cuuint32_t)kBM};
  const cuuint32_t box_vt[3] = {32, D, 1};
  if (!make_map_f32(&mq, qr, dq3, sq2, box_rows) || !make_map_f32(&mk, Nk > 0 ? kr : qr, dk3, sk2, box_rows) ||
      !make_map_f32(&mv, Nk > 0 ? (const void*)vt : qr, dv3, sv2, box_vt))
    return FA_ERR_CUDA;
  auto kern = fa_fwd_kernel<D, true, kKindTF32>;
  const int smem = FwdCfg<D, kKindTF32>::kSmemBytes;
  if (set_smem(kern, smem) != cudaSuccess) return FA_ERR_CUDA;
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  kern<<<std::min((int)units64, sms), kFwdThreads, smem, st>>>(mq, mk, mv, mq, prm);  // fp32 O: per-lane stores
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                 int Nk, int d, float scale, int causal, const int32_t* cu_seqlens, fa_dtype in_dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (in_dtype != FA_BF16 && in_dtype != FA_F32 && in_dtype != FA_TF32) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (in_dtype == FA_TF32 && (d != 64 || cu_seqlens != nullptr)) return FA_ERR_UNSUPPORTED;
  const bool varlen = cu_seqlens != nullptr;
  if (varlen) {
    if (Nq != Nk) return FA_ERR_INVALID_ARG;
    if (B > kMaxVarlenB || (int64_t)Nq > (int64_t)kMaxVarlenT * kUnitRows) return FA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return FA_ERR_INVALID_ARG;
  }
  const int64_t rows_q = varlen ? (int64_t)Nq : (int64_t)B * Nq;
  const int64_t rows_k = varlen ? (int64_t)Nk : (int64_t)B * Nk;
  if (rows_q >= (int64_t(1) << 31) || rows_k >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Nq == 0) return FA_OK;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (in_dtype == FA_TF32) return fwd_tf32(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, scale, causal, workspace,
                                           workspace_bytes, st);
  const void *qb = q, *kb = k, *vb = v;
  if (in_dtype == FA_F32) {
    const size_t need = fa_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, in_dtype, varlen ? 1 : 0);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
    const size_t nq = (size_t)rows_q * Hq * d, nk = (size_t)rows_k * Hkv * d;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    __nv_bfloat16* q16 = reinterpret_cast<__nv_bfloat16*>(w);
    __nv_bfloat16* k16 = reinterpret_cast<__nv_bfloat16*>(w + align_up(nq * 2, 256));
    __nv_bfloat16* v16 = reinterpret_cast<__nv_bfloat16*>(w + align_up(nq * 2, 256) + align_up(nk * 2, 256));
    const int sms = std::max(sm_count_cached(), 1);
    cast_f32_bf16_kernel<<<sms * 4, 256, 0, st>>>(static_cast<const float*>(q), q16, nq);
    if (nk > 0) {
      cast_f32_bf16_kernel<<<sms * 4, 256, 0, st>>>(static_cast<const float*>(k), k16, nk);
      cast_f32_bf16_kernel<<<sms * 4, 256, 0, st>>>(static_cast<const float*>(v), v16, nk);
    }
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    qb = q16;
    kb = k16;
    vb = v16;
  }

  FwdParams prm{};
  prm.o = o;
  prm.lse = lse;
  prm.cu = cu_seqlens;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Nq = Nq;
  prm.Nk = Nk;
  prm.causal = causal ? 1 : 0;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  prm.o_scale = 1.f;
  const int64_t units64 = fwd_units(prm, varlen, rows_q);
  if (units64 >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  const int units = (int)units64;
  const bool f32out = in_dtype == FA_F32;
  // rows_k may be 0 (no keys); the map still needs a non-zero extent
  const int64_t rk = std::max<int64_t>(rows_k, 1);
  if (d == 64)
    return f32out ? launch_fwd<64, true>(qb, kb, vb, prm, rows_q, rk, units, st)
                  : launch_fwd<64, false>(qb, kb, vb, prm, rows_q, rk, units, st);
  return f32out ? launch_fwd<128, true>(qb, kb, vb, prm, rows_q, rk, units, st)
                : launch_fwd<128, false>(qb, kb, vb, prm, rows_q, rk, units, st);
}

size_t fa_fwd_fp8_workspace_size(int B, int Hkv, int Nk, int d) {
  if (B <= 0 || Hkv <= 0 || Nk <= 0 || d != 128) return 0;
  const size_t pad = (size_t)(Nk + 15) / 16 * 16;
  return align_up((size_t)B * Hkv * d * pad, 256);
}

fa_status fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                     int Nq, int Nk, int d, float scale, float descale_q, float descale_k, float descale_v,
                     int causal, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
  for (float x : {scale, descale_q, descale_k, descale_v})
    if (!(x > 0.f) || !std::isfinite(x)) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  const int64_t rows_q = (int64_t)B * Nq, rows_k = (int64_t)B * Nk;
  if (rows_q >= (int64_t(1) << 31) || rows_k >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Nq == 0) return FA_OK;
  const int pad = (Nk + 15) / 16 * 16;
  const size_t need = fa_fwd_fp8_workspace_size(B, Hkv, Nk, d);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* vt = static_cast<uint8_t*>(workspace);
  if (Nk > 0) {
    dim3 g((pad + 63) / 64, Hkv, B);
    transpose_v_e4m3_kernel<<<g, 256, 0, st>>>(static_cast<const uint8_t*>(v), vt, Nk, Hkv, pad);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  FwdParams prm{};
  prm.o = o;
  prm.lse = lse;
  prm.cu = nullptr;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Nq = Nq;
  prm.Nk = Nk;
  prm.causal = causal ? 1 : 0;
  prm.tau = (float)((double)scale * descale_q * descale_k * 1.4426950408889634074);
  prm.o_scale = descale_v;
  const int64_t units64 = fwd_units(prm, false, rows_q);
  if (units64 >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  const cuuint64_t dq3[3] = {128, (cuuint64_t)Hq, (cuuint64_t)rows_q};
  const cuuint64_t sq2[2] = {128, (cuuint64_t)Hq * 128};
  const cuuint64_t dk3[3] = {128, (cuuint64_t)Hkv, (cuuint64_t)std::max<int64_t>(rows_k, 1)};
  const cuuint64_t sk2[2] = {128, (cuuint64_t)Hkv * 128};
  const cuuint64_t dv3[3] = {(cuuint64_t)std::max(pad, 16), 128, (cuuint64_t)B * Hkv};
  const cuuint64_t sv2[2] = {(cuuint64_t)std::max(pad, 16), (cuuint64_t)std::max(pad, 16) * 128};
  const cuuint32_t box_rows[3] = {128, 1, (cuuint32_t)kBM};
  const cuuint32_t box_vt[3] = {(cuuint32_t)kBN, 128, 1};
  if (!make_map_u8(&mq, q, dq3, sq2, box_rows) || !make_map_u8(&mk, k, dk3, sk2, box_rows) ||
      !make_map_u8(&mv, Nk > 0 ? (const void*)vt : k, dv3, sv2, box_vt))
    return FA_ERR_CUDA;
  CUtensorMap mo = mq;
  prm.o_tma = make_map_o(&mo, o, 128, Hq, rows_q) ? 1 : 0;
  auto kern = fa_fwd_kernel<128, false, kKindFP8>;
  const int smem = FwdCfg<128, kKindFP8>::kSmemBytes;
  if (set_smem(kern, smem) != cudaSuccess) return FA_ERR_CUDA;
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  const int units = (int)units64;
  kern<<<std::min(units, sms), kFwdThreads, smem, st>>>(mq, mk, mv, mo, prm);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd_qkvpacked(const void* qkv, void* o, float* lse, int B, int H, int N, int d, float scale, int causal,
                           const int32_t* cu_seqlens, void* stream) {
  if (!qkv || !o) return FA_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if (B < 0 || H <= 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const bool varlen = cu_seqlens != nullptr;
  if (varlen) {
    if (B > kMaxVarlenB || (int64_t)N > (int64_t)kMaxVarlenT * kUnitRows) return FA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return FA_ERR_INVALID_ARG;
  }
  const int64_t rows = varlen ? (int64_t)N : (int64_t)B * N;
  if (rows >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return FA_OK;
  FwdParams prm{};
  prm.o = o;
  prm.lse = lse;
  prm.cu = cu_seqlens;
  prm.B = B;
  prm.Hq = H;
  prm.Hkv = H;
  prm.G = 1;
  prm.Nq = N;
  prm.Nk = N;
  prm.causal = causal ? 1 : 0;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  prm.o_scale = 1.f;
  const int64_t units64 = fwd_units(prm, varlen, rows);
  if (units64 >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(qkv);
  const int64_t hd = (int64_t)H * d, stride = 3 * hd;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    return launch_fwd<64, false>(base, base + hd, base + 2 * hd, prm, rows, rows, (int)units64, st, stride, stride);
  return launch_fwd<128, false>(base, base + hd, base + 2 * hd, prm, rows, rows, (int)units64, st, stride, stride);
}

size_t fa_decode_workspace_size(int B, int Hq, int Lmax, int d, int split_len) {
  if (B <= 0 || Hq <= 0 || Lmax <= 0 || d <= 0 || split_len <= 0) return 0;
  const size_t ns = (size_t)((Lmax + split_len - 1) / split_len);
  const size_t parts = (size_t)B * Hq * ns;
  return align_up(parts * d * 4, 256) + align_up(parts * 2 * 4, 256);
}

fa_status fa_decode(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens, void* o,
                    float* lse, int B, int Hq, int Hkv, int Lmax, int d, float scale, int split_len,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !kcache || !vcache || !o) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Lmax <= 0 || split_len <= 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (seqlens && (reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (split_len % kDecKeys != 0) return FA_ERR_UNSUPPORTED;
  if ((int64_t)B * Lmax >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  const int nsplit = (Lmax + split_len - 1) / split_len;
  if (nsplit > 65535 || Hkv > 65535 || B > 65535) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_decode_workspace_size(B, Hq, Lmax, d, split_len);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  const size_t parts = (size_t)B * Hq * nsplit;
  DecParams prm{};
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.seqlens = seqlens;
  prm.o = static_cast<__nv_bfloat16*>(o);
  prm.lse = lse;
  prm.ws_acc = static_cast<float*>(workspace);
  prm.ws_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align_up(parts * d * 4, 256));
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Lmax = Lmax;
  prm.split_len = split_len;
  prm.nsplit = nsplit;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? launch_decode<64>(kcache, vcache, prm, st) : launch_decode<128>(kcache, vcache, prm, st);
}

size_t fa_decode_paged_workspace_size(int B, int Hq, int Hkv, int max_pages_per_seq, int page_size, int d,
                                      int split_len) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || max_pages_per_seq <= 0 || page_size <= 0 || d <= 0 || split_len <= 0)
    return 0;
  const int64_t lmax = (int64_t)max_pages_per_seq * page_size;
  if (lmax >= (int64_t(1) << 31)) return 0;
  return fa_decode_workspace_size(B, Hq, (int)lmax, d, split_len);  // the split partials
}

fa_status fa_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                          const int32_t* seqlens, void* o, float* lse, int B, int Hq, int Hkv, int num_pages,
                          int page_size, int max_pages_per_seq, int d, float scale, int split_len, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!q || !k_pages || !v_pages || !block_table || !seqlens || !o) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) != 0 || (reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || split_len <= 0)
    return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if ((page_size & (page_size - 1)) != 0) return FA_ERR_UNSUPPORTED;
  if (page_size < 16) return FA_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (split_len % kDecKeys != 0) return FA_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page_size >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  const int64_t lmax = (int64_t)max_pages_per_seq * page_size;
  if (lmax >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  const int nsplit = (int)((lmax + split_len - 1) / split_len);
  if (nsplit > 65535 || Hkv > 65535 || B > 65535) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_decode_paged_workspace_size(B, Hq, Hkv, max_pages_per_seq, page_size, d, split_len);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  const size_t parts = (size_t)B * Hq * nsplit;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecParams prm{};
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.seqlens = seqlens;
  prm.o = static_cast<__nv_bfloat16*>(o);
  prm.lse = lse;
  prm.ws_acc = reinterpret_cast<float*>(ws);
  prm.ws_ml = reinterpret_cast<float*>(ws + align_up(parts * d * 4, 256));
  prm.block_table = block_table;
  prm.max_pages = max_pages_per_seq;
  prm.page_shift = __builtin_ctz((unsigned)page_size);
  prm.page_box = std::min(page_size, kDecKeys);
  prm.num_pages = num_pages;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Lmax = (int)lmax;
  prm.split_len = split_len;
  prm.nsplit = nsplit;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? launch_decode_paged<64>(k_pages, v_pages, prm, st)
                 : launch_decode_paged<128>(k_pages, v_pages, prm, st);
}

size_t fa_bwd_workspace_size(int B, int Hq, int Nq, int d) {
  if (B <= 0 || Hq <= 0 || Nq <= 0 || d <= 0) return 0;
  const size_t pad = (size_t)(Nq + kBwdTile - 1) / kBwdTile * kBwdTile;
  return 2 * align_up((size_t)B * Hq * pad * 4, 256) + align_up((size_t)B * Nq * Hq * d * 4, 256);
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                 void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const int64_t rows_q = (int64_t)B * Nq, rows_k = (int64_t)B * Nk;
  if (rows_q >= (int64_t(1) << 31) || rows_k >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (B == 0 || (Nq == 0 && Nk == 0)) return FA_OK;
  const size_t need = fa_bwd_workspace_size(B, Hq, Nq, d);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return FA_ERR_WORKSPACE;
  BwdParams prm{};
  const int pad = (Nq + kBwdTile - 1) / kBwdTile * kBwdTile;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.lse2 = reinterpret_cast<float*>(ws);
  prm.dvec = reinterpret_cast<float*>(ws + align_up((size_t)B * Hq * pad * 4, 256));
  prm.dq_acc = reinterpret_cast<float*>(ws + 2 * align_up((size_t)B * Hq * pad * 4, 256));
  prm.o = static_cast<const __nv_bfloat16*>(o);
  prm.dout = static_cast<const __nv_bfloat16*>(dout);
  prm.lse = lse;
  prm.dq = static_cast<__nv_bfloat16*>(dq);
  prm.dk = static_cast<__nv_bfloat16*>(dk);
  prm.dv = static_cast<__nv_bfloat16*>(dv);
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Nq = Nq;
  prm.Nk = Nk;
  prm.NqPad = pad;
  prm.causal = causal ? 1 : 0;
  prm.scale = scale;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (Nq == 0) {
    // no query: every gradient is zero
    if (cudaMemsetAsync(dk, 0, (size_t)rows_k * Hkv * d * 2, st) != cudaSuccess ||
        cudaMemsetAsync(dv, 0, (size_t)rows_k * Hkv * d * 2, st) != cudaSuccess)
      return FA_ERR_CUDA;
    return FA_OK;
  }
  return d == 64 ? launch_bwd<64>(q, k, v, prm, st) : launch_bwd<128>(q, k, v, prm, st);
}

// Varlen backward: the tile bound and the workspace carve (tile prefix sums, two row vectors,
// the fp32 dq accumulator).
static int64_t bwd_varlen_ntiles(int B, int total) { return std::max<int64_t>(1, ((int64_t)total + 127 * (int64_t)B) / kBwdTile); }

size_t fa_bwd_varlen_workspace_size(int B, int Hq, int total, int d) {
  if (B <= 0 || Hq <= 0 || total <= 0 || d <= 0) return 0;
  const size_t vec = (size_t)Hq * bwd_varlen_ntiles(B, total) * kBwdTile * 4;
  return align_up((size_t)(B + 1) * 4, 256) + 2 * align_up(vec, 256) + align_up((size_t)total * Hq * d * 4, 256);
}

fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                        void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int total, int d, float scale,
                        int causal, const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || total < 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (B == 0 || total == 0) return FA_OK;
  const int64_t ntiles = bwd_varlen_ntiles(B, total);
  if (ntiles * kBwdTile >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_bwd_varlen_workspace_size(B, Hq, total, d);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  const size_t vec = align_up((size_t)Hq * ntiles * kBwdTile * 4, 256);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  BwdParams prm{};
  prm.tiles = reinterpret_cast<int32_t*>(ws);
  ws += align_up((size_t)(B + 1) * 4, 256);
  prm.lse2 = reinterpret_cast<float*>(ws);
  prm.dvec = reinterpret_cast<float*>(ws + vec);
  prm.dq_acc = reinterpret_cast<float*>(ws + 2 * vec);
  prm.o = static_cast<const __nv_bfloat16*>(o);
  prm.dout = static_cast<const __nv_bfloat16*>(dout);
  prm.lse = lse;
  prm.dq = static_cast<__nv_bfloat16*>(dq);
  prm.dk = static_cast<__nv_bfloat16*>(dk);
  prm.dv = static_cast<__nv_bfloat16*>(dv);
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.Nq = total;
  prm.Nk = total;
  prm.NqPad = 0;
  prm.causal = causal ? 1 : 0;
  prm.scale = scale;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  prm.cu = cu_seqlens;
  prm.ntiles = (int)ntiles;
  prm.total = total;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? launch_bwd<64>(q, k, v, prm, st) : launch_bwd<128>(q, k, v, prm, st);
}

fa_status fa_last_device_error(void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // one host thread at a time uses g_error_taken
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  take_error_word_kernel<<<1, 1, 0, st>>>();
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return FA_ERR_CUDA;
  unsigned int w = 0;
  if (cudaMemcpyFromSymbol(&w, g_error_taken, sizeof(w)) != cudaSuccess) return FA_ERR_CUDA;
  if (w & kErrTimeout) return FA_ERR_TIMEOUT;
  if (w & kErrSmem) return FA_ERR_CUDA;
  if (w != 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// Self-test of the bounded waits: one barrier that nothing arrives on.
namespace fa {
namespace {

__global__ void selftest_wait_kernel() {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_barrier_init();
  }
  __syncthreads();
  // phase 0 never completes: the wait gives up after its limit, records the timeout and returns
  if (threadIdx.x == 0) (void)mbar_wait(&bar, 0);
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_selftest_wait_timeout(void* stream) {
  fa::selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>();
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------
// fa_decode_noalloc: fa_decode with its scratch in a static device array, for callers that
// cannot allocate device memory (see include/fa.h).
namespace fa {
namespace {

// The split partials of fa_decode_noalloc.  In host code this name is only a stand-in for
// the symbol; its device address comes from cudaGetSymbolAddress (per device).
static __device__ __align__(256) unsigned char g_decode_noalloc_scratch[FA_DECODE_NOALLOC_SCRATCH_BYTES];

std::mutex g_noalloc_mu;
void* g_noalloc_ptr[64] = {};

// Device address of the scratch array on the current device, looked up once per device.
fa_status noalloc_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_decode_noalloc_scratch) != cudaSuccess || p == nullptr) return FA_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_decode_noalloc(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens,
                                       void* o, float* lse, int B, int Hq, int Hkv, int Lmax, int d, float scale,
                                       int split_len, void* stream) {
  // Argument checks of fa_decode, without a workspace: a valid non-empty problem stops at the
  // workspace check (nothing launched); anything else is returned as is.
  const fa_status pre = fa_decode(q, kcache, vcache, seqlens, o, lse, B, Hq, Hkv, Lmax, d, scale, split_len,
                                  nullptr, 0, stream);
  if (pre != FA_ERR_WORKSPACE) return pre;
  if (fa_decode_workspace_size(B, Hq, Lmax, d, split_len) > (size_t)FA_DECODE_NOALLOC_SCRATCH_BYTES)
    return FA_ERR_WORKSPACE;
  void* scratch = nullptr;
  const fa_status st = fa::noalloc_scratch(&scratch);
  if (st != FA_OK) return st;
  return fa_decode(q, kcache, vcache, seqlens, o, lse, B, Hq, Hkv, Lmax, d, scale, split_len, scratch,
                   (size_t)FA_DECODE_NOALLOC_SCRATCH_BYTES, stream);
}

// ---------------------------------------------------------------------------------------
// Rotary positions.
namespace fa {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T, int D>
fa_status launch_rope(RopeParams prm, cudaStream_t st) {
  constexpr int V = RopeVec<T>::N, heads_at_once = 32 / (D / (2 * V));
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  // Runs of heads: one for each row when the rows alone fill the GPU, else as many as give
  // each SM 32 warps, down to the heads that a warp covers at once.
  const int nh = prm.heads[0] + prm.heads[1], groups = (nh + heads_at_once - 1) / heads_at_once;
  const long long want = std::max(1ll, (sms * 32ll) / prm.rows);
  const int per = (int)((groups + std::min<long long>(want, groups) - 1) / std::min<long long>(want, groups));
  prm.per_chunk = per * heads_at_once;
  prm.chunks = (nh + prm.per_chunk - 1) / prm.per_chunk;
  const unsigned blocks = (unsigned)((prm.rows * prm.chunks + 7) / 8);
  const auto kern = prm.interleaved         ? fa_rope_vec_kernel<T, D, true>
                    : prm.rot / 2 % V == 0 ? fa_rope_vec_kernel<T, D, false>
                                           : fa_rope_kernel<T, D>;
  return launch_early(kern, blocks, 256, 0, st, prm) ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_rope_frequencies(double* freqs, int rot_dim, double theta, fa_rope_scaling scaling,
                                         double factor, double original_len, double low, double high) {
  if (!freqs || rot_dim <= 0 || rot_dim % 2 != 0) return FA_ERR_INVALID_ARG;
  if (!(theta > 0.0) || !std::isfinite(theta)) return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_NONE && scaling != FA_ROPE_LINEAR && scaling != FA_ROPE_NTK && scaling != FA_ROPE_BANDS)
    return FA_ERR_INVALID_ARG;
  if (scaling != FA_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor))) return FA_ERR_INVALID_ARG;
  if (scaling == FA_ROPE_BANDS && (!(original_len > 0.0) || !std::isfinite(original_len) || !(low < high) ||
                                   !std::isfinite(low) || !std::isfinite(high)))
    return FA_ERR_INVALID_ARG;
  const double two_pi = 6.28318530717958647693;
  if (scaling == FA_ROPE_NTK && rot_dim > 2) theta *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == FA_ROPE_LINEAR) w /= factor;
    if (scaling == FA_ROPE_BANDS) {
      const double turns = original_len * w / two_pi;
      const double keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
      w *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = w;
  }
  return FA_OK;
}

extern "C" fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                             const double* freqs, long long rows, int period, int Hq, int Hk, int d, int rot_dim,
                             int interleaved, float amplitude, int backward, fa_dtype dtype, long long q_stride,
                             long long k_stride, long long q_out_stride, long long k_out_stride, void* stream) {
  if (rows < 0 || Hq <= 0 || Hk < 0 || !q || !q_out || !freqs) return FA_ERR_INVALID_ARG;
  if (Hk > 0 && (!k || !k_out)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_F32) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return FA_ERR_INVALID_ARG;
  if (!positions && period <= 0) return FA_ERR_INVALID_ARG;
  if (!aligned4(positions) || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot_dim <= 0 || rot_dim > d || rot_dim % 2 != 0) return FA_ERR_INVALID_ARG;
  const int es = dtype == FA_BF16 ? 2 : 4;
  const void* ptrs[4] = {q, q_out, Hk > 0 ? k : q, Hk > 0 ? k_out : q_out};
  const long long strides[4] = {q_stride, q_out_stride, Hk > 0 ? k_stride : q_stride,
                                Hk > 0 ? k_out_stride : q_out_stride};
  for (int i = 0; i < 4; ++i) {
    const int h = i < 2 ? Hq : std::max(Hk, 1);
    if (!aligned16(ptrs[i]) || strides[i] < (long long)h * d || strides[i] * es % 16 != 0) return FA_ERR_INVALID_ARG;
  }
  // written in place only over the very rows that were read
  if ((q == q_out && q_stride != q_out_stride) || (Hk > 0 && k == k_out && k_stride != k_out_stride))
    return FA_ERR_INVALID_ARG;
  if (rows >= (1ll << 31) || (long long)Hq + Hk > 65535) return FA_ERR_UNSUPPORTED;
  if (rows == 0) return FA_OK;
  RopeParams prm{};
  prm.x[0] = q;
  prm.x[1] = k;
  prm.y[0] = q_out;
  prm.y[1] = k_out;
  prm.xs[0] = q_stride;
  prm.xs[1] = k_stride;
  prm.ys[0] = q_out_stride;
  prm.ys[1] = k_out_stride;
  prm.heads[0] = Hq;
  prm.heads[1] = Hk;
  prm.positions = positions;
  prm.freqs = freqs;
  prm.rows = rows;
  prm.period = period;
  prm.rot = rot_dim;
  prm.interleaved = interleaved ? 1 : 0;
  prm.backward = backward ? 1 : 0;
  prm.amplitude = amplitude;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == FA_BF16)
    return d == 64 ? launch_rope<__nv_bfloat16, 64>(prm, st) : launch_rope<__nv_bfloat16, 128>(prm, st);
  return d == 64 ? launch_rope<float, 64>(prm, st) : launch_rope<float, 128>(prm, st);
}

// ---------------------------------------------------------------------------------------
// The paged cache in e4m3.
namespace fa {
namespace {

// What the append and the decode over the e4m3 cache check alike.
fa_status check_cache8(const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale,
                       const int32_t* block_table, const int32_t* seqlens, int B, int Hkv, int num_pages,
                       int page_size, int max_pages, int scale_block, int d) {
  if (!k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seqlens) return FA_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned4(k_scale) || !aligned4(v_scale) ||
      !aligned4(block_table) || !aligned4(seqlens))
    return FA_ERR_INVALID_ARG;
  if (B < 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0 || scale_block <= 0)
    return FA_ERR_INVALID_ARG;
  if ((page_size & (page_size - 1)) != 0 || page_size < 16) return FA_ERR_UNSUPPORTED;
  if ((scale_block & (scale_block - 1)) != 0 || scale_block < 16 || scale_block > 256 || scale_block > page_size)
    return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page_size >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  // (room for positions rounded up to a chunk)
  if ((int64_t)max_pages * page_size > (int64_t(1) << 31) - 1024) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

template <int D>
fa_status launch_append(const AppendParams& prm, cudaStream_t st) {
  const int upc = kAppendCta / append_warps<D>(prm.sb_shift);
  const dim3 grid((unsigned)(prm.cu ? (prm.total >> prm.sb_shift) + 2ll * prm.B : prm.B),
                  (unsigned)((prm.Hkv + upc - 1) / upc));
  return launch_early(fa_cache_append_kernel<D>, grid, kAppendCta * 32, 0, st, prm) ? FA_OK : FA_ERR_CUDA;
}

// What a unit costs beside its chunks, in chunks (128 sequences of up to 600 rows, 8 K/V heads, d = 128,
// without it: 42 us instead of 28 for 8 query rows, 271 instead of 139 for 40; 64 of up to 4K, 8 rows: 57
// instead of 50).
constexpr int kDec8Lead = 4, kDec8TcLead = 10;
// Query rows of a unit: the 8 columns of a tensor-core product, or its 16 rows, where that holds them
// (8 rows over 8 sequences of 32K: 90 us instead of 100 as 16); else the kernel on tcgen05 products with 64
// (d = 128: 40 rows, 8 sequences of up to 32K, in 104 us instead of 211 with 64 rows in registers), or
// registers for 32 or 64 (d = 64, where a cache row is too short for those products' 128 rows).
int dec8_tile(int64_t rows, int d) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 && d == 64 ? 32 : 64; }
// K/V heads of a unit, as a shift: one where the query rows fill more than a tile (the products,
// not the loads, take the time then, and one head's queries are all that shared memory holds).
int dec8_heads(int tile, int Hkv) { return tile > 16 ? 0 : Hkv % 4 == 0 ? 2 : Hkv % 2 == 0 ? 1 : 0; }
// One wave of CTAs (where no device is present, the number of the B200's).
int dec8_ctas(int tile, int d) {
  const int sms = sm_count_cached();
  const int per_sm = tile == 8    ? Dec8Cfg<128>::kCtas
                     : tile == 16 ? (d == 64 ? Dec8WideCfg<64, 1, 1>::kCtas : Dec8WideCfg<128, 1, 1>::kCtas)
                     : tile == 32 ? Dec8WideCfg<64, 2, 1>::kCtas
                                  : 1;
  return (sms > 0 ? sms : 148) * per_sm;
}

bool dec8_maps(CUtensorMap (&maps)[2], const void* kp, const void* vp, int d, const Dec8Params& prm) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)prm.num_pages << prm.page_shift, (cuuint64_t)prm.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)prm.Hkv * d, (cuuint64_t)d};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)prm.box, 1u << prm.hs}, estr[3] = {1, 1, 1};
  for (int w = 0; w < 2; ++w)
    if (enc(&maps[w], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w ? vp : kp), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

template <int D, int R>
fa_status launch_decode_fp8_merge(const Dec8Params& prm, int ctas, cudaStream_t st) {
  // No unit can be cut where the longest sequence that the table holds is short.
  if ((prm.cap - 1 >> (7 - prm.hs)) + 1 <= kDec8Whole) return FA_OK;
  // The merge starts on the SMs that the last CTAs leave and waits there for their results.
  const int items = std::min(prm.rows, R) << prm.hs, gx = prm.by_unit ? prm.B * prm.units : ctas;
  const bool wide = (int64_t)gx * items <= 8ll * ctas;
  const dim3 grid(gx, wide ? items : (items + 7) / 8);
  const auto kern = wide ? fa_decode_fp8_combine_kernel<D, R, true> : fa_decode_fp8_combine_kernel<D, R, false>;
  return launch_early(kern, grid, 256, 0, st, prm) ? FA_OK : FA_ERR_CUDA;
}

template <class C, int D, class K>
fa_status launch_decode_fp8(K kern, const void* kp, const void* vp, const Dec8Params& prm, cudaStream_t st) {
  CUtensorMap maps[2];
  if (!dec8_maps(maps, kp, vp, D, prm)) return FA_ERR_CUDA;
  static std::atomic<uint64_t> smem_set{0};  // a bit for each device
  if (!set_smem_once(kern, C::kSmem, smem_set)) return FA_ERR_CUDA;
  const int ctas = dec8_ctas(C::kRows, D);
  if (!launch_early(kern, ctas, C::kThreads, C::kSmem, st, maps[0], maps[1], prm)) return FA_ERR_CUDA;
  return launch_decode_fp8_merge<D, C::kRows>(prm, ctas, st);
}

template <int D>
fa_status launch_decode_fp8_narrow(const void* kp, const void* vp, const Dec8Params& prm, cudaStream_t st) {
  return launch_decode_fp8<Dec8Cfg<D>, D>(fa_decode_fp8_kernel<D>, kp, vp, prm, st);
}

template <int D, int MT, int RG>
fa_status launch_decode_fp8_wide(const void* kp, const void* vp, const Dec8Params& prm, cudaStream_t st) {
  return launch_decode_fp8<Dec8WideCfg<D, MT, RG>, D>(fa_decode_fp8_wide_kernel<D, MT, RG>, kp, vp, prm, st);
}

fa_status launch_decode_fp8_tc(const void* kp, const void* vp, const Dec8Params& prm, cudaStream_t st) {
  return launch_decode_fp8<Dec8TcCfg, Dec8TcCfg::D>(fa_decode_fp8_tc_kernel, kp, vp, prm, st);
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_cache_append_fp8(const void* k, const void* v, const int32_t* cu_seqlens,
                                         const int32_t* block_table, const int32_t* seqlens, void* k_pages,
                                         void* v_pages, float* k_scale, float* v_scale, int B, int total, int Hkv,
                                         int num_pages, int page_size, int max_pages_per_seq, int scale_block, int d,
                                         void* stream) {
  const fa_status ok = check_cache8(k_pages, v_pages, k_scale, v_scale, block_table, seqlens, B, Hkv, num_pages,
                                    page_size, max_pages_per_seq, scale_block, d);
  if (ok != FA_OK) return ok;
  if (total < 0 || (!cu_seqlens && total != B) || !aligned4(cu_seqlens)) return FA_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return FA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
  AppendParams prm{};
  prm.src[0] = static_cast<const __nv_bfloat16*>(k);
  prm.src[1] = static_cast<const __nv_bfloat16*>(v);
  prm.pages[0] = static_cast<uint8_t*>(k_pages);
  prm.pages[1] = static_cast<uint8_t*>(v_pages);
  prm.scales[0] = k_scale;
  prm.scales[1] = v_scale;
  prm.cu = cu_seqlens;
  prm.block_table = block_table;
  prm.seqlens = seqlens;
  prm.B = B;
  prm.total = total;
  prm.Hkv = Hkv;
  prm.num_pages = num_pages;
  prm.page_shift = __builtin_ctz((unsigned)page_size);
  prm.max_pages = max_pages_per_seq;
  prm.sb_shift = __builtin_ctz((unsigned)scale_block);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? launch_append<64>(prm, st) : launch_append<128>(prm, st);
}

extern "C" size_t fa_decode_paged_fp8_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0) return 0;
  // two parts per CTA (sums, then m and l) and a descriptor per CTA
  const int tile = dec8_tile((int64_t)Nq * (Hq / Hkv), d);
  const size_t ctas = (size_t)dec8_ctas(tile, d);
  const size_t slots = (2 * ctas * tile) << dec8_heads(tile, Hkv);
  return align_up(slots * d * 4, 256) + align_up(slots * 8, 256) + align_up(ctas * 16, 256);
}

extern "C" fa_status fa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                                         const float* k_scale, const float* v_scale, const int32_t* block_table,
                                         const int32_t* seqlens, void* o, float* lse, int B, int Nq, int Hq, int Hkv,
                                         int num_pages, int page_size, int max_pages_per_seq, int scale_block, int d,
                                         float scale, void* workspace, size_t workspace_bytes, void* stream) {
  const fa_status ok = check_cache8(k_pages, v_pages, k_scale, v_scale, block_table, seqlens, B, Hkv, num_pages,
                                    page_size, max_pages_per_seq, scale_block, d);
  if (ok != FA_OK) return ok;
  if (Nq < 0 || Hq <= 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Nq == 0) return FA_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o) || !aligned4(lse)) return FA_ERR_INVALID_ARG;
  if (Nq > 65535 || Hq > 65535) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_decode_paged_fp8_workspace_size(B, Nq, Hq, Hkv, d);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  const int64_t rows = (int64_t)Nq * (Hq / Hkv);
  if (rows * Hkv >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  Dec8Params prm{};
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.scales[0] = k_scale;
  prm.scales[1] = v_scale;
  prm.block_table = block_table;
  prm.seqlens = seqlens;
  prm.o = static_cast<__nv_bfloat16*>(o);
  prm.lse = lse;
  prm.B = B;
  prm.Nq = Nq;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.num_pages = num_pages;
  prm.page_shift = __builtin_ctz((unsigned)page_size);
  prm.sb_shift = __builtin_ctz((unsigned)scale_block);
  prm.max_pages = max_pages_per_seq;
  prm.tau = (float)((double)scale * 1.4426950408889634074);
  prm.rows = (int)rows;
  const int tile = dec8_tile(rows, d);
  prm.tiles = (prm.rows + tile - 1) / tile;
  prm.hs = dec8_heads(tile, Hkv);
  prm.box = std::min(page_size, kDec8Keys >> prm.hs);
  const size_t ctas = (size_t)dec8_ctas(tile, d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.ws_acc = reinterpret_cast<float*>(ws);
  const size_t slots = (2 * ctas * tile) << prm.hs;
  ws += align_up(slots * d * 4, 256);
  prm.ws_ml = reinterpret_cast<float2*>(ws);
  prm.ws_desc = reinterpret_cast<int4*>(ws + align_up(slots * 8, 256));
  prm.cap = (int)((int64_t)max_pages_per_seq * page_size);
  const int64_t units = (int64_t)(Hkv >> prm.hs) * prm.tiles;
  // positions among all chunks are 32-bit in the kernel
  prm.lead = tile == 64 && d == 128 ? kDec8TcLead : kDec8Lead;
  if (B * units * (((prm.cap - 1) >> (7 - prm.hs)) + 1 + prm.lead) >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  prm.units = (int)units;
  prm.by_unit = B * units <= (int64_t)ctas;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d == 64)
    return tile == 8    ? launch_decode_fp8_narrow<64>(k_pages, v_pages, prm, st)
           : tile == 16 ? launch_decode_fp8_wide<64, 1, 1>(k_pages, v_pages, prm, st)
           : tile == 32 ? launch_decode_fp8_wide<64, 2, 1>(k_pages, v_pages, prm, st)
                        : launch_decode_fp8_wide<64, 2, 2>(k_pages, v_pages, prm, st);
  return tile == 8    ? launch_decode_fp8_narrow<128>(k_pages, v_pages, prm, st)
         : tile == 16 ? launch_decode_fp8_wide<128, 1, 1>(k_pages, v_pages, prm, st)
                      : launch_decode_fp8_tc(k_pages, v_pages, prm, st);
}

// ---------------------------------------------------------------------------------------
// Pages of a cache.
namespace fa {
namespace {

fa_status check_pages(const fa_pool* pools, int n_pools, const int32_t* block_table, const int32_t* seqlens, int B,
                      int num_pages, int page_size, int max_pages) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return FA_ERR_INVALID_ARG;
  if (B < 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
  if (B > 0 && (!block_table || !seqlens || !aligned4(block_table) || !aligned4(seqlens))) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < n_pools; ++i)
    if (!pools[i].base || pools[i].page_bytes == 0) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < n_pools; ++i)
    if (pools[i].page_bytes >= (size_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  if ((page_size & (page_size - 1)) != 0 || n_pools > kMaxPools * kMaxLaunches) return FA_ERR_UNSUPPORTED;
  if (num_pages >= kFreeMark || (int64_t)max_pages * page_size >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status launch_copies(const fa_pool* pools, int n_pools, const int32_t* src, const int32_t* dst,
                        const int32_t* count, int32_t* tickets, cudaStream_t st) {
  const int sms = sm_count_cached();
  if (sms <= 0) return FA_ERR_CUDA;
  static std::atomic<uint64_t> smem_set{0};  // a bit for each device
  if (!set_smem_once(pages_copy_kernel, kCopySmem, smem_set)) return FA_ERR_CUDA;
  for (int at = 0; at < n_pools; at += kMaxPools) {
    PoolList list{};
    const int m = std::min(kMaxPools, n_pools - at);
    // pools whose pages are worth bulk copies first
    for (int turn = 0; turn < 2; ++turn) {
      for (int i = 0; i < m; ++i) {
        const fa_pool& pool = pools[at + i];
        const uintptr_t mis = reinterpret_cast<uintptr_t>(pool.base) | pool.page_bytes;
        const unsigned vec = (mis & 15) == 0 ? 16 : (mis & 3) == 0 ? 4 : 1, vpp = (unsigned)pool.page_bytes / vec;
        const bool bulk = vec == 16 && pool.page_bytes >= 4096;
        if (bulk != (turn == 0)) continue;
        const unsigned per = bulk ? kBulkBytes / 16 : kCopyVecs;  // vectors of an item
        const int k = list.n++;
        list.base[k] = static_cast<uint8_t*>(pool.base);
        list.vec[k] = (uint8_t)vec;
        list.vpp[k] = vpp;
        list.pages[k] = !bulk && vpp <= per / 2 ? per / vpp : 0;
        list.pieces[k] = (vpp + per - 1) / per;
      }
      if (turn == 0) list.bulk = list.n;
    }
    if (!launch_early(pages_copy_kernel, sms * 2, kCopyThreads + 32, kCopySmem, st, list, src, dst, count, tickets++))
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" size_t fa_pages_workspace_size(int num_pages, int B_out) {
  if (num_pages <= 0 || B_out < 0) return 0;
  return align_up((size_t)num_pages * 4, 256) + 256 +
         4 * align_up((size_t)std::max(num_pages / 2 + 1, B_out) * 4, 256);
}

extern "C" fa_status fa_pages_fork(const fa_pool* pools, int n_pools, const int32_t* block_table,
                                   const int32_t* seqlens, const int32_t* parent, int32_t* block_table_out,
                                   int32_t* seqlens_out, int32_t* free_pages, int32_t* n_free, int B, int B_out,
                                   int num_pages, int page_size, int max_pages_per_seq, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const fa_status ok = check_pages(pools, n_pools, block_table, seqlens, B, num_pages, page_size, max_pages_per_seq);
  if (ok != FA_OK) return ok;
  if (B_out < 0 || !free_pages || !n_free || !aligned4(free_pages) || !aligned4(n_free)) return FA_ERR_INVALID_ARG;
  if (B_out > 0 && (!parent || !block_table_out || !seqlens_out || !aligned4(parent) || !aligned4(block_table_out) ||
                    !aligned4(seqlens_out)))
    return FA_ERR_INVALID_ARG;
  if (B_out > 0 && (block_table_out == block_table || seqlens_out == seqlens)) return FA_ERR_INVALID_ARG;
  const size_t need = fa_pages_workspace_size(num_pages, B_out);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t list = align_up((size_t)std::max(num_pages / 2 + 1, B_out) * 4, 256);
  ForkParams prm{};
  prm.table = block_table;
  prm.lens = seqlens;
  prm.parent = parent;
  prm.table_out = block_table_out;
  prm.lens_out = seqlens_out;
  prm.free_pages = free_pages;
  prm.n_free = n_free;
  prm.mark = reinterpret_cast<int32_t*>(ws);
  ws += align_up((size_t)num_pages * 4, 256);
  prm.count = reinterpret_cast<int32_t*>(ws);
  prm.tickets = prm.count + 4;
  prm.counts = prm.tickets + kMaxLaunches;
  ws += 256;
  prm.rank = reinterpret_cast<int32_t*>(ws);
  prm.src = reinterpret_cast<int32_t*>(ws + list);
  prm.dst = reinterpret_cast<int32_t*>(ws + 2 * list);
  prm.B = B;
  prm.R = B_out;
  prm.max_pages = max_pages_per_seq;
  prm.page_shift = __builtin_ctz((unsigned)page_size);
  prm.num_pages = num_pages;
  if (!launch_early(fork_plan_kernel, kPlanCtas, kPlanThreads, 0, st, prm)) return FA_ERR_CUDA;
  return launch_copies(pools, n_pools, prm.src, prm.dst, prm.count, prm.tickets, st);
}

extern "C" fa_status fa_pages_compact(const fa_pool* pools, int n_pools, const int32_t* block_table,
                                      const int32_t* seqlens, int32_t* block_table_out, int32_t* n_live, int B,
                                      int num_pages, int page_size, int max_pages_per_seq, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const fa_status ok = check_pages(pools, n_pools, block_table, seqlens, B, num_pages, page_size, max_pages_per_seq);
  if (ok != FA_OK) return ok;
  if (!n_live || !aligned4(n_live)) return FA_ERR_INVALID_ARG;
  if (B > 0 && (!block_table_out || !aligned4(block_table_out) || block_table_out == block_table))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_pages_workspace_size(num_pages, 0);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return FA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t list = align_up((size_t)(num_pages / 2 + 1) * 4, 256);
  CompactParams prm{};
  prm.table = block_table;
  prm.lens = seqlens;
  prm.table_out = block_table_out;
  prm.n_live = n_live;
  prm.mark = reinterpret_cast<int32_t*>(ws);
  ws += align_up((size_t)num_pages * 4, 256);
  prm.count = reinterpret_cast<int32_t*>(ws);
  prm.tickets = prm.count + 4;
  prm.counts = prm.tickets + kMaxLaunches;
  ws += 256;
  prm.src = reinterpret_cast<int32_t*>(ws);
  prm.dst = reinterpret_cast<int32_t*>(ws + list);
  prm.B = B;
  prm.max_pages = max_pages_per_seq;
  prm.page_shift = __builtin_ctz((unsigned)page_size);
  prm.num_pages = num_pages;
  if (!launch_early(compact_plan_kernel, kPlanCtas, kPlanThreads, 0, st, prm)) return FA_ERR_CUDA;
  return launch_copies(pools, n_pools, prm.src, prm.dst, prm.count, prm.tickets, st);
}

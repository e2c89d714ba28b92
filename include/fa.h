/* Exact IO-aware attention for NVIDIA B200 (sm_100a): C ABI.
 *
 * Exact attention O = softmax(Q K^T * scale) V with the per-row logsumexp, computed tile by
 * tile with the online-softmax running max m and sum l, so the N x N score and probability
 * matrices never reach device memory; its backward; and the decode step over a KV cache:
 *
 *   fa_fwd     the tiled forward ("FlashAttention notes", section 3 "Tiling" and section 4
 *              "Online Softmax": m_new = max(m1, m2), l_new = e^(m1-m_new) l1 + e^(m2-m_new) l2;
 *              "LLM basics: from Attention to FlashAttention", chapter 3 section 5), with
 *              causal masking (same tutorial, chapter 1 section 7), grouped-query heads
 *              (chapter 2 section 7) and variable-length packed batches ("FlashAttention-3
 *              (FA-3)", section 2 feature table: MQA, GQA, variable-length).
 *   fa_decode  single-token decode over a KV cache, split along the cache; the partial
 *              results are merged with the same m/l rule ("FlashAttention-3 (FA-3)",
 *              section 4 "FlashDecoding"; "FlashAttention notes", section 4).
 *   fa_decode_paged  the same decode over a paged cache addressed through a block table.
 *   fa_bwd     the backward of fa_fwd by recomputation from the saved logsumexp;
 *              fa_bwd_varlen the same over packed variable-length sequences.
 *   fa_fwd_qkvpacked  fa_fwd reading q, k, v from one packed [.., 3, H, d] tensor.
 *   fa_fwd_fp8 the forward on e4m3 inputs with per-tensor scales.
 *   fa_rope    rotary positions of q and k, and their gradients, around fa_fwd and fa_bwd.
 *   fa_cache_append_fp8, fa_decode_paged_fp8  a paged cache held in e4m3 with a scale for each
 *              block of tokens and head: writing new K/V rows, and attention over it.
 *   fa_pages_fork, fa_pages_compact  sharing, copying, freeing and moving the pages of a paged
 *              cache of any element type.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library never
 *     allocates or frees device memory and never synchronises, except in
 *     fa_last_device_error.  Every launch is asynchronous on `stream` (a cudaStream_t
 *     passed as void*; NULL is the legacy default stream).
 *   - Tensors are contiguous with the head dimension d innermost (fa_fwd_qkvpacked reads
 *     its three slices with a row stride of 3 H d).  bf16 is IEEE bfloat16.
 *   - Arguments are validated on the host before anything is launched; a rejected call
 *     returns FA_ERR_INVALID_ARG or FA_ERR_UNSUPPORTED and touches no memory.
 *   - A failed launch returns FA_ERR_CUDA.  A device-side wait that exceeded its time
 *     limit (it never should) is recorded on the device and reported by
 *     fa_last_device_error as FA_ERR_TIMEOUT; the kernel then returns instead of hanging.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_EXPORT __attribute__((visibility("default")))
#else
#define FA_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad scale */
  FA_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. d not in {64, 128}) */
  FA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the *_workspace_size() value */
  FA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
  FA_ERR_TIMEOUT = 5      /* a device wait gave up (reported by fa_last_device_error) */
} fa_status;

typedef enum { FA_BF16 = 0, FA_F32 = 1, FA_TF32 = 2 } fa_dtype;

/* Forward attention.
 *
 * Fixed length (cu_seqlens == NULL):
 *   q [B, Nq, Hq, d], k and v [B, Nk, Hkv, d], o [B, Nq, Hq, d], lse [B, Hq, Nq].
 * Variable length (cu_seqlens != NULL, device int32 [B+1]):
 *   Nq == Nk == total packed rows; q and o [total, Hq, d], k and v [total, Hkv, d],
 *   lse [Hq, total]; sequence b owns rows [cu_seqlens[b], cu_seqlens[b+1]) of q, k and v and
 *   attends only within itself.  cu_seqlens must start at or above 0, never decrease and end
 *   at or below total; it is read on the device only, and one that breaks this is found
 *   there: nothing is read or written and fa_last_device_error reports FA_ERR_INVALID_ARG.
 *   Rows outside every sequence are not written.  B <= 1024.
 *
 * in_dtype FA_BF16: q, k, v, o are bf16.  FA_F32: q, k, v are fp32, rounded to bf16 (nearest
 *   even) into the workspace first, and o is written as fp32 (fixed or variable length).
 *   FA_TF32: q, k,
 *   v are fp32, rounded to tf32 (10 mantissa bits, nearest even) into the workspace, and the
 *   products run on the tf32 tensor-core path with P kept in fp32; o fp32; fixed length,
 *   d = 64 (the workspace also holds v transposed).
 * Accumulation is fp32; P is rounded to bf16 before the P*V product.
 * scale: the score multiplier, > 0 (1/sqrt(d) in "LLM basics", chapter 1 section 3).
 * causal: query i of a sequence with nq queries and nk keys sees keys j <= i + nk - nq
 *   (bottom-right aligned; the usual lower triangle when nq == nk).  A row that sees no
 *   key gets o = 0 and lse = -inf.
 * lse: natural-log logsumexp of the scaled scores, fp32; may be NULL.
 * Hq must be a multiple of Hkv; query head h uses key/value head h / (Hq / Hkv).
 * d must be 64 or 128.  q, k, v, o must be 16-byte aligned.
 * workspace: device memory of at least fa_fwd_workspace_size(...) bytes (may be NULL when
 *   that size is 0).
 */
FA_EXPORT fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                 int Nq, int Nk, int d, float scale, int causal, const int32_t* cu_seqlens, fa_dtype in_dtype,
                 void* workspace, size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_fwd_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d, fa_dtype in_dtype, int varlen);

/* FP8 forward ("Attention is All You Need부터 FlashAttention-3까지", FlashAttention-3 section:
 * FP8 support for higher throughput; "FlashAttention-3 (FA-3)", section 2 feature table: FP8):
 * q, k, v are e4m3 (OCP FP8, stored one byte each) with per-tensor dequantisation factors:
 * the value of an element is (its e4m3 value) * descale_x.  Computes the same O and lse as
 * fa_fwd for the dequantised inputs: S = q k^T on the e4m3 tensor-core path (fp32
 * accumulation, exact products), softmax in fp32, P rounded to e4m3 (nearest even, values
 * <= 256 by the lazy rescale) for the P V product, l summed from the unrounded P; O is written
 * as bf16, lse as in fa_fwd.  Fixed length; d must be 128.
 * q [B, Nq, Hq, 128], k and v [B, Nk, Hkv, 128] (bytes), o [B, Nq, Hq, 128] bf16,
 * lse [B, Hq, Nq] fp32 (may be NULL).  Same causal rule and head grouping as fa_fwd.
 * workspace: at least fa_fwd_fp8_workspace_size(B, Hkv, Nk, 128) bytes; it receives a
 * transposed copy of v ([B, Hkv, 128, Nk rounded up to 16]) so that both operands of P V are
 * K-major. */
FA_EXPORT fa_status fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                               int Hkv, int Nq, int Nk, int d, float scale, float descale_q, float descale_k,
                               float descale_v, int causal, void* workspace, size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_fwd_fp8_workspace_size(int B, int Hkv, int Nk, int d);

/* Forward attention on a packed qkv tensor (the flash_attn_qkvpacked_func interface of
 * "Attention is All You Need부터 FlashAttention-3까지", section "practical implementation: using
 * FlashAttention in PyTorch", whose example is qkv [2, 2048, 3, 12, 64], causal): q, k and v
 * are the three slices of qkv [B, N, 3, H, d] bf16 (fixed length) or [total, 3, H, d] with
 * cu_seqlens (variable length, as in fa_fwd, N = total rows).  H query heads and H key/value
 * heads; o [B, N, H, d] (or [total, H, d]) bf16; lse as in fa_fwd (may be NULL).  Read in
 * place through strided tensor maps: no copy, no workspace.  d 64 or 128; qkv and o 16-byte
 * aligned. */
FA_EXPORT fa_status fa_fwd_qkvpacked(const void* qkv, void* o, float* lse, int B, int H, int N, int d, float scale,
                                     int causal, const int32_t* cu_seqlens, void* stream);

/* Backward of fa_fwd (fixed length): gradients dq, dk, dv of o = attention(q, k, v) for an
 * upstream gradient dout of o ("FlashAttention notes", section 5.2 backward: P is rebuilt on
 * chip from q, k and the saved logsumexp instead of being stored; dV = P^T dO, dP = dO V^T,
 * dS = P o (dP - D) with D_i = sum_c dO_ic O_ic, dQ = scale dS K, dK = scale dS^T Q).
 *
 * q, o, dout, dq [B, Nq, Hq, d] bf16; k, v, dk, dv [B, Nk, Hkv, d] bf16; lse [B, Hq, Nq] fp32,
 * the natural-log logsumexp that fa_fwd wrote for (q, k, v, scale, causal), and o the output
 * it wrote.  Same scale, causal rule and head grouping as fa_fwd; dk and dv sum over the
 * query heads of each group.  Accumulation is fp32; P and dS are rounded to bf16 for the
 * tensor-core products; dq, dk, dv are rounded to bf16 (nearest even).
 * d 64 or 128; pointers 16-byte aligned (lse 4-byte aligned).
 * workspace: at least fa_bwd_workspace_size(B, Hq, Nq, d) bytes (two padded fp32 row vectors
 * and an fp32 dq accumulator); its contents need not be initialised. */
FA_EXPORT fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                           const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk,
                           int d, float scale, int causal, void* workspace, size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_bwd_workspace_size(int B, int Hq, int Nq, int d);

/* Backward of fa_fwd on packed variable-length sequences ("FlashAttention-3 (FA-3)", feature
 * table: variable-length batches; the method is that of fa_bwd, within each sequence).
 *
 * Sequence b owns rows [cu_seqlens[b], cu_seqlens[b+1]) of q, o, dout, dq [total, Hq, d] and
 * of k, v, dk, dv [total, Hkv, d] (bf16); lse [Hq, total] fp32 as fa_fwd wrote it with the same
 * cu_seqlens.  No attention, and so no gradient, crosses a sequence boundary; causal is
 * within each sequence.  cu_seqlens: device int32 [B + 1], starting at or above 0, never
 * decreasing, ending at or below total; a cu_seqlens that breaks this is found on the
 * device: nothing is computed and fa_last_device_error reports FA_ERR_INVALID_ARG.  Rows
 * outside every sequence get dq = 0 and their dk, dv are not written; rows of q, k, v and
 * dout past cu_seqlens[B] are read as padding of the last sequence's last tile and must hold
 * finite values.
 * d 64 or 128; pointers 16-byte aligned (lse and cu_seqlens 4-byte aligned).
 * workspace: at least fa_bwd_varlen_workspace_size(B, Hq, total, d) bytes (tile prefix sums,
 * two fp32 row vectors padded per sequence to 128-row tiles, an fp32 dq accumulator); its
 * contents need not be initialised. */
FA_EXPORT fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                  const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int total,
                                  int d, float scale, int causal, const int32_t* cu_seqlens, void* workspace,
                                  size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_bwd_varlen_workspace_size(int B, int Hq, int total, int d);

/* Split-KV decode: one query token per sequence against its KV cache.
 *
 * q [B, Hq, d] bf16; kcache and vcache [B, Lmax, Hkv, d] bf16; o [B, Hq, d] bf16;
 * lse [B, Hq] fp32 (may be NULL); seqlens: device int32 [B] with 0 <= seqlens[b] <= Lmax,
 * or NULL meaning every sequence holds Lmax tokens.  Sequence b attends (non-causally) to
 * cache rows j < seqlens[b]; an empty sequence gets o = 0 and lse = -inf.
 * The cache is cut into splits of split_len rows (a multiple of 64); each split's partial
 * (m, l, unnormalised acc) goes to the workspace and a second kernel merges them with the
 * m/l rule.  Hq / Hkv <= 16.  d must be 64 or 128.  Pointers 16-byte aligned.
 */
FA_EXPORT fa_status fa_decode(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens, void* o,
                    float* lse, int B, int Hq, int Hkv, int Lmax, int d, float scale, int split_len,
                    void* workspace, size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_decode_workspace_size(int B, int Hq, int Lmax, int d, int split_len);

/* Largest scratch, in bytes, that fa_decode_noalloc can use (16 MiB). */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES (16u << 20)

/* fa_decode for callers that cannot allocate device memory.
 *
 * Some callers have no way to call cudaMalloc on this path: a host program that only
 * receives its input and output buffers from someone else (a plugin inside another
 * framework's memory pool), or a latency-critical loop where an allocation, which can
 * synchronise the device, is not allowed.  This entry point takes the same arguments as
 * fa_decode minus the workspace and allocates nothing.  The pages describe no such entry
 * point; it exists only for these callers.
 *
 * Scratch: the split partials live in one static device array of
 * FA_DECODE_NOALLOC_SCRATCH_BYTES in this library, which every GPU that loads the library
 * holds until the process exits.  Problems whose scratch need (fa_decode_workspace_size)
 * exceeds it are rejected with FA_ERR_WORKSPACE before anything is launched; the decode
 * workload B=8, Hq=64, d=128, cache 32768, splits of 1024 needs about 8.7 MB.
 * No part of the scratch has to start at zero: every partial the merge reads is written by
 * the same call.  All calls share the array, so calls that overlap on the GPU (on
 * different streams, or on one stream from different threads without ordering) race and
 * give wrong results; order them on one stream.
 * The first call on each device looks up the array's device address (with that device
 * current) and caches it; make that first call before any stream capture.  The cached
 * address belongs to that device's context: a process that resets the device
 * (cudaDeviceReset) or otherwise tears its primary context down must not call this entry
 * point on that device again, since the library's device memory may then sit elsewhere.
 * Other arguments, results and errors are those of fa_decode. */
FA_EXPORT fa_status fa_decode_noalloc(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens,
                                      void* o, float* lse, int B, int Hq, int Hkv, int Lmax, int d, float scale,
                                      int split_len, void* stream);

/* Split-KV decode over a paged KV cache ("LLM basics: from Attention to FlashAttention",
 * chapter 2 section 8, PagedAttention: fixed-size pages of the cache, mapped from each
 * sequence's logical pages by a block table); the splits are merged as in fa_decode.
 *
 * q [B, Hq, d] bf16; k_pages and v_pages [num_pages, page_size, Hkv, d] bf16 (the page
 * pool); block_table: device int32 [B, max_pages_per_seq], entry (b, t) = the physical page
 * holding tokens t*page_size .. (t+1)*page_size - 1 of sequence b; seqlens: device int32 [B],
 * required, 0 <= seqlens[b] <= max_pages_per_seq * page_size (larger values are clamped).
 * Only the first ceil(seqlens[b] / page_size) entries of row b are read; pages may be
 * shared between sequences and appear in any order.  o [B, Hq, d] bf16; lse [B, Hq] fp32
 * (may be NULL).  Token j of sequence b takes part iff j < seqlens[b]; an empty sequence gets
 * o = 0 and lse = -inf.  Rows of a page beyond a sequence's length may hold anything
 * (NaN included): they are masked and never multiply into o.
 * page_size: a power of two >= 16.  split_len: a multiple of 64.  Hq / Hkv <= 16; d 64 or
 * 128; q, the pages and o 16-byte aligned; block_table and seqlens 4-byte aligned;
 * num_pages * page_size < 2^31.
 * A block-table entry outside [0, num_pages) is read as page 0 and recorded on the device;
 * fa_last_device_error then returns FA_ERR_INVALID_ARG.
 * workspace: at least fa_decode_paged_workspace_size(...) bytes (the split partials); its
 * contents need not be initialised.  Calls sharing a workspace must not overlap on the GPU. */
FA_EXPORT fa_status fa_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* block_table, const int32_t* seqlens, void* o, float* lse, int B,
                                    int Hq, int Hkv, int num_pages, int page_size, int max_pages_per_seq, int d,
                                    float scale, int split_len, void* workspace, size_t workspace_bytes,
                                    void* stream);

FA_EXPORT size_t fa_decode_paged_workspace_size(int B, int Hq, int Hkv, int max_pages_per_seq, int page_size, int d,
                                                int split_len);

/* Rotary positions.  The first rot_dim columns of every head of q and k turn in pairs: pair i
 * < rot_dim / 2 of a row at position p turns by the angle p * freqs[i],
 *   y_a = amplitude (x_a cos - x_b sin),  y_b = amplitude (x_b cos + x_a sin),
 * with (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) if `interleaved`; the other columns are
 * copied.  backward != 0 gives the gradient: x is the gradient of y, y that of x (the same
 * formula with -sin).  Angles are reduced in fp64, so far positions lose nothing; their sines and
 * cosines (within 1.5 * 2^-24, and 2^-51 of the angle) and the products are fp32, rounded once to the
 * element type.
 *
 * q [rows, Hq, d], k [rows, Hk, d] (Hk may be 0: q alone), each row's heads dense and rows
 * q_stride / k_stride elements apart (Hq * d when dense; 3 H d for q and k inside a packed
 * [rows, 3, H, d] tensor); q_out, k_out likewise.  An output may be its input (same pointer and
 * stride); it must not overlap either input in another way.  Element type FA_BF16 or FA_F32.
 * positions: device int32 [rows], any values (negative ones turn backwards), or NULL: row r has
 * position r % period (period = the length of each sequence of a fixed-length batch).
 * freqs: device fp64 [rot_dim / 2], radians per position (fa_rope_frequencies gives the usual
 * ones).  d 64 or 128; rot_dim even, 2 .. d.  Pointers 16-byte aligned (positions 4, freqs 8),
 * strides multiples of 16 bytes.  No workspace. */
FA_EXPORT fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                            const double* freqs, long long rows, int period, int Hq, int Hk, int d, int rot_dim,
                            int interleaved, float amplitude, int backward, fa_dtype dtype, long long q_stride,
                            long long k_stride, long long q_out_stride, long long k_out_stride, void* stream);

/* How fa_rope_frequencies stretches positions for contexts longer than the trained one. */
typedef enum {
  FA_ROPE_NONE = 0,   /* w_i = theta^(-2 i / rot_dim) */
  FA_ROPE_LINEAR = 1, /* w_i / factor */
  FA_ROPE_NTK = 2,    /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta (rot_dim > 2) */
  FA_ROPE_BANDS = 3   /* by the turns over original_len positions, r_i = original_len w_i / 2 pi: above `high`
                         kept, below `low` divided by factor, linear in r_i in between */
} fa_rope_scaling;

/* Writes rot_dim / 2 frequencies to HOST memory (fp64), to be copied to the device once. */
FA_EXPORT fa_status fa_rope_frequencies(double* freqs, int rot_dim, double theta, fa_rope_scaling scaling,
                                        double factor, double original_len, double low, double high);

/* Appends K and V rows to a paged cache held in e4m3 with a scale for each block.
 *
 * k, v [total, Hkv, d] bf16: the new rows of all sequences, sequence b owning rows
 * [cu_seqlens[b], cu_seqlens[b+1]) (device int32 [B + 1], starting at or above 0, never
 * decreasing, ending at or below total), or one row each (cu_seqlens NULL, total == B).
 * k_pages, v_pages [num_pages, page_size, Hkv, d] e4m3 bytes; k_scale, v_scale fp32
 * [num_pages, Hkv, page_size / scale_block]: the value of an element is (its e4m3 value) * (the
 * scale of its block of scale_block rows and head).  block_table int32 [B, max_pages_per_seq] as
 * in fa_decode_paged; seqlens: device int32 [B], lengths INCLUDING the new rows (the same array
 * then goes to fa_decode_paged_fp8): n new rows of sequence b become its tokens seqlens[b] - n ..
 * seqlens[b] - 1.
 * A block that receives rows gets the scale max(s, s'), with s' the least power of two (at least
 * 2^-126) for which no new |x| exceeds 448 s' (0 if all are 0) and s its scale so far if it
 * already holds rows of the sequence, else 0; new elements are stored as x / scale, rounded to
 * nearest even; if the scale grew, the rows held already are multiplied by old / new and rounded
 * again.  A new row that is not finite makes the scale of its blocks NaN.  Rows past a
 * sequence's end, and scales of blocks that receive nothing, are left as they were.
 * Pages that receive rows must belong to one sequence each (fa_pages_fork sees to that).
 * A sequence whose offsets or length cannot be used (see above; n > seqlens[b]; seqlens[b] >
 * max_pages_per_seq * page_size) and a page outside [0, num_pages) are skipped and recorded:
 * fa_last_device_error then returns FA_ERR_INVALID_ARG.
 * page_size a power of two >= 16; scale_block a power of two, 16 .. min(256, page_size); d 64 or
 * 128; k, v and the pages 16-byte aligned, the rest 4; num_pages * page_size < 2^31.  No
 * workspace. */
FA_EXPORT fa_status fa_cache_append_fp8(const void* k, const void* v, const int32_t* cu_seqlens,
                                        const int32_t* block_table, const int32_t* seqlens, void* k_pages,
                                        void* v_pages, float* k_scale, float* v_scale, int B, int total, int Hkv,
                                        int num_pages, int page_size, int max_pages_per_seq, int scale_block, int d,
                                        void* stream);

/* Decode over a paged cache in e4m3 (as fa_cache_append_fp8 writes it), for one or more new
 * query tokens per sequence.
 *
 * q [B, Nq, Hq, d] bf16: the Nq newest tokens of each sequence, whose K and V rows are in the
 * cache already; o likewise; lse [B, Hq, Nq] fp32 (may be NULL).  Query i of sequence b sees
 * cache rows j <= seqlens[b] - Nq + i (every row for Nq = 1); a query that sees no row gets o = 0
 * and lse = -inf.  Cache, scales, block_table and seqlens as in fa_cache_append_fp8
 * (scales 0 .. 2^120 or NaN; the append writes no larger ones for finite rows); lengths below 0
 * count as 0, larger ones than max_pages_per_seq * page_size as that.  Rows past a sequence's end may
 * hold anything; a NaN code or scale makes NaN of what attends to it, and of nothing else.  An entry of
 * the table outside [0, num_pages) is read as page 0 and recorded (FA_ERR_INVALID_ARG from
 * fa_last_device_error).
 * The stored values are exact in the products and all sums are fp32.  P times the V scale is rounded
 * to fp16 relative to a value within 2^6 of its largest.  For more than 16 query rows of a K/V head
 * (Nq * Hq / Hkv) and d = 128, q is the sum of two e4m3 terms (8 bits, like bf16; 2^-17 of a row's
 * largest element at the least), and V scales outside 2^-100 .. 2^100 lose accuracy.  o is rounded to
 * bf16.
 * Hq a multiple of Hkv; d 64 or 128; sizes as in fa_cache_append_fp8, and B * Hkv *
 * (max_pages_per_seq * page_size + 1408) * (Nq * (Hq / Hkv) / 64, rounded up) < 2^38 suffices for what
 * is counted in 32 bits (FA_ERR_UNSUPPORTED beyond).  workspace: at least
 * fa_decode_paged_fp8_workspace_size(...) bytes (with the call's device current), 16-byte aligned, not
 * initialised; calls that share one must not overlap on the GPU.  o and lse must not overlap the
 * inputs. */
FA_EXPORT fa_status fa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                                        const float* k_scale, const float* v_scale, const int32_t* block_table,
                                        const int32_t* seqlens, void* o, float* lse, int B, int Nq, int Hq, int Hkv,
                                        int num_pages, int page_size, int max_pages_per_seq, int scale_block, int d,
                                        float scale, void* workspace, size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_decode_paged_fp8_workspace_size(int B, int Nq, int Hq, int Hkv, int d);

/* One array of a paged cache (K or V pages or their scales, of one layer): num_pages pages of
 * page_bytes bytes each, in device memory. */
typedef struct {
  void* base;
  size_t page_bytes;
} fa_pool;

/* Forks, drops and reorders the sequences of a paged cache.
 *
 * New sequence i (of B_out) continues sequence parent[i] (device int32 [B_out], entries in
 * [0, B), or -1 for an empty sequence): seqlens_out[i] = seqlens[parent[i]], and its row of
 * block_table_out names the same pages, except that a last page that is not full is kept by the
 * first new sequence that ends in it only, and copied to a free page for every other one (for
 * all of them if some new sequence holds that page full).  Sequences without a successor are
 * dropped.  A page is in use if it is among the first ceil(len / page_size) entries of a new
 * sequence; free_pages [num_pages] receives the other pages in ascending order, without those
 * that the copies took (the lowest ones, in the order of the new sequences), then -1;
 * n_free [1] their number.  Entries of a row past the sequence's pages become -1.
 * Pages are copied in every pool of `pools` (a HOST array of n_pools; any element types; 0 pools:
 * tables only; at most 4096; pages under 2^31 bytes).  block_table [B, max_pages_per_seq] and
 * block_table_out [B_out, max_pages_per_seq], all device int32; outputs must not overlap inputs.
 * page_size is a power of two.
 * Recorded for fa_last_device_error (FA_ERR_INVALID_ARG): a parent outside [-1, B) (taken as
 * -1), a length that is negative or past the table (taken as 0), an entry outside [0, num_pages)
 * (passed on, never copied), and too few free pages (those new sequences become empty; pages that only
 * they name are in no list then, and come back with the next fork or compaction).
 * workspace: at least fa_pages_workspace_size(num_pages, B_out) bytes, 16-byte aligned, not
 * initialised; calls that share one must not overlap on the GPU. */
FA_EXPORT fa_status fa_pages_fork(const fa_pool* pools, int n_pools, const int32_t* block_table,
                                  const int32_t* seqlens, const int32_t* parent, int32_t* block_table_out,
                                  int32_t* seqlens_out, int32_t* free_pages, int32_t* n_free, int B, int B_out,
                                  int num_pages, int page_size, int max_pages_per_seq, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Moves the pages in use to the front of the pool: of n_live pages in use (n_live [1], device),
 * the k-th at or past index n_live is copied to the k-th free page before it, in every pool, and
 * block_table_out names the new places (-1 past each sequence's pages).  Pages from n_live on are
 * free afterwards.  Arguments, checks and workspace (fa_pages_workspace_size(num_pages, 0)) as in
 * fa_pages_fork. */
FA_EXPORT fa_status fa_pages_compact(const fa_pool* pools, int n_pools, const int32_t* block_table,
                                     const int32_t* seqlens, int32_t* block_table_out, int32_t* n_live, int B,
                                     int num_pages, int page_size, int max_pages_per_seq, void* workspace,
                                     size_t workspace_bytes, void* stream);

FA_EXPORT size_t fa_pages_workspace_size(int num_pages, int B_out);

/* Takes the device-side error record (read and cleared in one atomic exchange, on `stream`),
 * waits for `stream`, and returns FA_ERR_TIMEOUT if any kernel of this library recorded a
 * device-side timeout since the previous call, else FA_ERR_CUDA if a kernel found its shared
 * memory carve-out too small, else FA_ERR_INVALID_ARG if a kernel recorded an invalid
 * device-side input (a block-table entry out of range, a cu_seqlens that fa_fwd or
 * fa_bwd_varlen cannot use, what fa_cache_append_fp8 and the fa_pages calls name); FA_ERR_CUDA if the
 * stream reports an error; else FA_OK.
 * The record is shared by all kernels of the library on the device (all streams); a timeout
 * stops only the kernel whose wait ran out, and later launches run normally whether or not
 * the record has been taken. */
FA_EXPORT fa_status fa_last_device_error(void* stream);

/* Test support for the failure detection: launches one kernel whose single wait can never be
 * satisfied (nothing arrives on its barrier).  The wait is bounded like every wait of the
 * library: after its time limit (4 s) it records a timeout and the kernel returns, so nothing
 * hangs and the context stays usable; the next fa_last_device_error reports FA_ERR_TIMEOUT. */
FA_EXPORT fa_status fa_selftest_wait_timeout(void* stream);

/* Static description of a status code. */
FA_EXPORT const char* fa_status_string(fa_status s);

/* Number of streaming multiprocessors of the current device (0 on failure); the forward
 * kernel's persistent grid uses one CTA per SM. */
FA_EXPORT int fa_device_sm_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */

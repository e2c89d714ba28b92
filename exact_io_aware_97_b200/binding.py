"""ctypes binding of libfa.so: the functions of include/fa.h under the same names.

Argument marshalling only: pointers come from torch tensors (``data_ptr()``) or plain
integers, the stream defaults to torch's current stream, and a non-OK status raises
``FaError``.  Every step of the computation runs in the library's CUDA kernels; there is no
fallback.  If libfa.so is missing this module raises on first use.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_BF16, FA_F32, FA_TF32 = 0, 1, 2
FA_ROPE_NONE, FA_ROPE_LINEAR, FA_ROPE_NTK, FA_ROPE_BANDS = range(4)

EXPORTED = ("fa_fwd", "fa_fwd_workspace_size", "fa_decode", "fa_decode_workspace_size", "fa_decode_noalloc",
            "fa_decode_paged", "fa_decode_paged_workspace_size", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_varlen",
            "fa_bwd_varlen_workspace_size", "fa_fwd_qkvpacked",
            "fa_fwd_fp8", "fa_fwd_fp8_workspace_size", "fa_selftest_wait_timeout",
            "fa_rope", "fa_rope_frequencies", "fa_cache_append_fp8", "fa_decode_paged_fp8",
            "fa_decode_paged_fp8_workspace_size", "fa_pages_fork", "fa_pages_compact", "fa_pages_workspace_size",
            "fa_last_device_error", "fa_status_string", "fa_device_sm_count")
FA_DECODE_NOALLOC_SCRATCH_BYTES = 16 << 20


class FaPool(ctypes.Structure):
    """fa_pool: one array of a paged cache."""
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so (once).  Raises if the CUDA library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libfa.so not found at {path}; build it with `python -m exact_io_aware_97_b200.build`")
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, i, vp, sz, vp]
    L.fa_fwd.restype = i
    L.fa_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    L.fa_fwd_workspace_size.restype = sz
    L.fa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
    L.fa_decode.restype = i
    L.fa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    L.fa_decode_noalloc.restype = i
    L.fa_decode_workspace_size.argtypes = [i, i, i, i, i]
    L.fa_decode_workspace_size.restype = sz
    L.fa_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, sz, vp]
    L.fa_decode_paged.restype = i
    L.fa_decode_paged_workspace_size.argtypes = [i, i, i, i, i, i, i]
    L.fa_decode_paged_workspace_size.restype = sz
    L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, f, f, f, i, vp, sz, vp]
    L.fa_fwd_fp8.restype = i
    L.fa_fwd_fp8_workspace_size.argtypes = [i, i, i, i]
    L.fa_fwd_fp8_workspace_size.restype = sz
    L.fa_fwd_qkvpacked.argtypes = [vp, vp, vp, i, i, i, i, f, i, vp, vp]
    L.fa_fwd_qkvpacked.restype = i
    L.fa_bwd.argtypes = [vp] * 9 + [i] * 6 + [f, i, vp, sz, vp]
    L.fa_bwd.restype = i
    L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    L.fa_bwd_workspace_size.restype = sz
    L.fa_bwd_varlen.argtypes = [vp] * 9 + [i] * 5 + [f, i, vp, vp, sz, vp]
    L.fa_bwd_varlen.restype = i
    L.fa_bwd_varlen_workspace_size.argtypes = [i, i, i, i]
    L.fa_bwd_varlen_workspace_size.restype = sz
    ll, db = ctypes.c_longlong, ctypes.c_double
    L.fa_rope.argtypes = [vp] * 6 + [ll] + [i] * 6 + [f, i, i] + [ll] * 4 + [vp]
    L.fa_rope.restype = i
    L.fa_rope_frequencies.argtypes = [vp, i, db, i, db, db, db, db]
    L.fa_rope_frequencies.restype = i
    L.fa_cache_append_fp8.argtypes = [vp] * 9 + [i] * 8 + [vp]
    L.fa_cache_append_fp8.restype = i
    L.fa_decode_paged_fp8.argtypes = [vp] * 9 + [i] * 9 + [f, vp, sz, vp]
    L.fa_decode_paged_fp8.restype = i
    L.fa_decode_paged_fp8_workspace_size.argtypes = [i] * 5
    L.fa_decode_paged_fp8_workspace_size.restype = sz
    L.fa_pages_fork.argtypes = [vp, i] + [vp] * 7 + [i] * 5 + [vp, sz, vp]
    L.fa_pages_fork.restype = i
    L.fa_pages_compact.argtypes = [vp, i] + [vp] * 4 + [i] * 4 + [vp, sz, vp]
    L.fa_pages_compact.restype = i
    L.fa_pages_workspace_size.argtypes = [i, i]
    L.fa_pages_workspace_size.restype = sz
    L.fa_selftest_wait_timeout.argtypes = [vp]
    L.fa_selftest_wait_timeout.restype = i
    L.fa_last_device_error.argtypes = [vp]
    L.fa_last_device_error.restype = i
    L.fa_status_string.argtypes = [i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_device_sm_count.argtypes = []
    L.fa_device_sm_count.restype = i
    _lib = L
    return L


def _ptr(x) -> Optional[int]:
    """Device address of a tensor argument (an int is taken as a raw address).  The library
    reads every tensor as a dense row-major block of device memory, so a host tensor or a
    strided view is refused here rather than handed to a kernel."""
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    if not x.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"expected a contiguous tensor, got strides {tuple(x.stride())} for shape {tuple(x.shape)}")
    return x.data_ptr() or None


def _ptr_i32(x, what: str) -> Optional[int]:
    """Device address of an int32 index tensor (offsets, lengths, block table): the kernels
    read these as int32, so another integer width would be misread as other offsets."""
    if x is not None and not isinstance(x, int) and str(x.dtype) != "torch.int32":
        raise ValueError(f"{what}: expected an int32 tensor, got {x.dtype}")
    return _ptr(x)


def _expect(t, shape, dtype: str, what: str) -> None:
    """A caller-provided output must have exactly the shape and dtype the kernels write."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or str(t.dtype) != dtype:
        raise ValueError(f"{what}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _same(what: str, *ts) -> None:
    """Tensors that the kernels read with one shape and one element type."""
    a = ts[0]
    for t in ts[1:]:
        if tuple(t.shape) != tuple(a.shape) or t.dtype != a.dtype:
            raise ValueError(f"{what}: shapes/dtypes differ: {tuple(a.shape)} {a.dtype} vs {tuple(t.shape)} {t.dtype}")


def _require(what: str, ok: bool, expected: str) -> None:
    """A relation between tensors that the kernels rely on: they size every read from q's
    batch and head dimension, so a smaller k or cache would be read past its end."""
    if not ok:
        raise ValueError(f"{what}: expected {expected}")


def _lengths(seqlens, B: int, what: str) -> None:
    """Per-sequence lengths are read as B int32 entries."""
    if seqlens is not None and not isinstance(seqlens, int):
        _require(what, seqlens.dim() == 1 and seqlens.numel() == B, f"{B} entries, got shape {tuple(seqlens.shape)}")


def _bf16(what: str, *ts) -> None:
    """Paths that read bf16 only (the backward, the decodes)."""
    for t in ts:
        if str(t.dtype) != "torch.bfloat16":
            raise ValueError(f"{what}: expected bf16 tensors, got {t.dtype}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        # the raw handle of torch.cuda.current_stream(), without building the Stream object where torch
        # has a function for that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None or not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream or None
        return raw(torch.cuda.current_device()) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FaError(status, where)


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, cu_seqlens=None, in_dtype=FA_BF16,
           workspace=None, workspace_bytes=0, stream=None) -> None:
    st = load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(Nq), int(Nk),
                       int(d), float(scale), int(bool(causal)), _ptr_i32(cu_seqlens, "cu_seqlens"), int(in_dtype), _ptr(workspace),
                       int(workspace_bytes), _stream(stream))
    _check(st, "fa_fwd")


def fa_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, in_dtype=FA_BF16, varlen=False) -> int:
    return int(load().fa_fwd_workspace_size(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(d), int(in_dtype),
                                            int(bool(varlen))))


def fa_decode(q, kcache, vcache, seqlens, o, lse, B, Hq, Hkv, Lmax, d, scale, split_len, workspace,
              workspace_bytes, stream=None) -> None:
    st = load().fa_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr_i32(seqlens, "seqlens"), _ptr(o), _ptr(lse), int(B), int(Hq),
                          int(Hkv), int(Lmax), int(d), float(scale), int(split_len), _ptr(workspace),
                          int(workspace_bytes), _stream(stream))
    _check(st, "fa_decode")


def fa_decode_noalloc(q, kcache, vcache, seqlens, o, lse, B, Hq, Hkv, Lmax, d, scale, split_len,
                      stream=None) -> None:
    """fa_decode with its scratch in the library's static device array (no allocation).
    For callers that cannot allocate device memory; calls that overlap on the GPU race, and
    the first call on a device should come before any stream capture (see include/fa.h)."""
    st = load().fa_decode_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr_i32(seqlens, "seqlens"), _ptr(o), _ptr(lse), int(B),
                                  int(Hq), int(Hkv), int(Lmax), int(d), float(scale), int(split_len),
                                  _stream(stream))
    _check(st, "fa_decode_noalloc")


def fa_decode_workspace_size(B, Hq, Lmax, d, split_len) -> int:
    return int(load().fa_decode_workspace_size(int(B), int(Hq), int(Lmax), int(d), int(split_len)))


def fa_decode_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, B, Hq, Hkv, num_pages, page_size,
                    max_pages_per_seq, d, scale, split_len, workspace, workspace_bytes, stream=None) -> None:
    st = load().fa_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr_i32(block_table, "block_table"), _ptr_i32(seqlens, "seqlens"), _ptr(o),
                                _ptr(lse), int(B), int(Hq), int(Hkv), int(num_pages), int(page_size),
                                int(max_pages_per_seq), int(d), float(scale), int(split_len), _ptr(workspace),
                                int(workspace_bytes), _stream(stream))
    _check(st, "fa_decode_paged")


def fa_decode_paged_workspace_size(B, Hq, Hkv, max_pages_per_seq, page_size, d, split_len) -> int:
    return int(load().fa_decode_paged_workspace_size(int(B), int(Hq), int(Hkv), int(max_pages_per_seq),
                                                     int(page_size), int(d), int(split_len)))


def fa_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, descale_q, descale_k, descale_v, causal, workspace,
               workspace_bytes, stream=None) -> None:
    st = load().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(Nq),
                           int(Nk), int(d), float(scale), float(descale_q), float(descale_k), float(descale_v),
                           int(bool(causal)), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "fa_fwd_fp8")


def fa_fwd_fp8_workspace_size(B, Hkv, Nk, d) -> int:
    return int(load().fa_fwd_fp8_workspace_size(int(B), int(Hkv), int(Nk), int(d)))


def fa_fwd_qkvpacked(qkv, o, lse, B, H, N, d, scale, causal, cu_seqlens=None, stream=None) -> None:
    st = load().fa_fwd_qkvpacked(_ptr(qkv), _ptr(o), _ptr(lse), int(B), int(H), int(N), int(d), float(scale),
                                 int(bool(causal)), _ptr_i32(cu_seqlens, "cu_seqlens"), _stream(stream))
    _check(st, "fa_fwd_qkvpacked")


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, workspace, workspace_bytes,
           stream=None) -> None:
    st = load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                       int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(d), float(scale), int(bool(causal)),
                       _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "fa_bwd")


def fa_bwd_workspace_size(B, Hq, Nq, d) -> int:
    return int(load().fa_bwd_workspace_size(int(B), int(Hq), int(Nq), int(d)))


def fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, total, d, scale, causal, cu_seqlens, workspace,
                  workspace_bytes, stream=None) -> None:
    st = load().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                              _ptr(dv), int(B), int(Hq), int(Hkv), int(total), int(d), float(scale),
                              int(bool(causal)), _ptr_i32(cu_seqlens, "cu_seqlens"), _ptr(workspace), int(workspace_bytes),
                              _stream(stream))
    _check(st, "fa_bwd_varlen")


def fa_bwd_varlen_workspace_size(B, Hq, total, d) -> int:
    return int(load().fa_bwd_varlen_workspace_size(int(B), int(Hq), int(total), int(d)))


def fa_rope(q, k, q_out, k_out, positions, freqs, rows, period, Hq, Hk, d, rot_dim, interleaved, amplitude, backward,
            dtype, q_stride, k_stride, q_out_stride, k_out_stride, stream=None) -> None:
    """q, k and the outputs as raw addresses or dense tensors; strides in elements between rows."""
    st = load().fa_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr_i32(positions, "positions"), _ptr(freqs),
                        int(rows), int(period), int(Hq), int(Hk), int(d), int(rot_dim), int(bool(interleaved)),
                        float(amplitude), int(bool(backward)), int(dtype), int(q_stride), int(k_stride),
                        int(q_out_stride), int(k_out_stride), _stream(stream))
    _check(st, "fa_rope")


def fa_rope_frequencies(rot_dim, theta=10000.0, scaling=FA_ROPE_NONE, factor=1.0, original_len=0.0, low=0.0,
                        high=0.0) -> list:
    """rot_dim / 2 angular frequencies as floats (host)."""
    buf = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    _check(load().fa_rope_frequencies(ctypes.cast(buf, ctypes.c_void_p), int(rot_dim), float(theta), int(scaling),
                                      float(factor), float(original_len), float(low), float(high)),
           "fa_rope_frequencies")
    return list(buf)


def fa_cache_append_fp8(k, v, cu_seqlens, block_table, seqlens, k_pages, v_pages, k_scale, v_scale, B, total, Hkv,
                        num_pages, page_size, max_pages_per_seq, scale_block, d, stream=None) -> None:
    st = load().fa_cache_append_fp8(_ptr(k), _ptr(v), _ptr_i32(cu_seqlens, "cu_seqlens"),
                                    _ptr_i32(block_table, "block_table"), _ptr_i32(seqlens, "seqlens"),
                                    _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), int(B), int(total),
                                    int(Hkv), int(num_pages), int(page_size), int(max_pages_per_seq),
                                    int(scale_block), int(d), _stream(stream))
    _check(st, "fa_cache_append_fp8")


def fa_decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, o, lse, B, Nq, Hq, Hkv,
                        num_pages, page_size, max_pages_per_seq, scale_block, d, scale, workspace, workspace_bytes,
                        stream=None) -> None:
    st = load().fa_decode_paged_fp8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                    _ptr_i32(block_table, "block_table"), _ptr_i32(seqlens, "seqlens"), _ptr(o),
                                    _ptr(lse), int(B), int(Nq), int(Hq), int(Hkv), int(num_pages), int(page_size),
                                    int(max_pages_per_seq), int(scale_block), int(d), float(scale), _ptr(workspace),
                                    int(workspace_bytes), _stream(stream))
    _check(st, "fa_decode_paged_fp8")


def fa_decode_paged_fp8_workspace_size(B, Nq, Hq, Hkv, d) -> int:
    return int(load().fa_decode_paged_fp8_workspace_size(int(B), int(Nq), int(Hq), int(Hkv), int(d)))


def _pool_array(pools, num_pages):
    """fa_pool array (address and page_bytes in turn) of tensors [num_pages, ...]; raw pairs pass
    through.  The caller keeps it for the call."""
    flat = array.array("Q")
    for n, t in enumerate(pools):
        if isinstance(t, tuple):
            flat.extend(t)
            continue
        if t.dim() < 1 or t.shape[0] != num_pages:
            raise ValueError(f"pool {n}: expected [{num_pages}, ...], got shape {tuple(t.shape)}")
        if not t.is_cuda or not t.is_contiguous():
            _ptr(t)  # says what is wrong
        flat.append(t.data_ptr())
        flat.append(t.nbytes // max(num_pages, 1))
    return flat


def _pool_ptr(flat) -> Optional[int]:
    return flat.buffer_info()[0] if flat else None


def fa_pages_fork(pools, block_table, seqlens, parent, block_table_out, seqlens_out, free_pages, n_free, B, B_out,
                  num_pages, page_size, max_pages_per_seq, workspace, workspace_bytes, stream=None) -> None:
    arr = _pool_array(pools, int(num_pages))
    st = load().fa_pages_fork(_pool_ptr(arr), len(pools), _ptr_i32(block_table, "block_table"), _ptr_i32(seqlens, "seqlens"),
                              _ptr_i32(parent, "parent"), _ptr_i32(block_table_out, "block_table_out"),
                              _ptr_i32(seqlens_out, "seqlens_out"), _ptr_i32(free_pages, "free_pages"),
                              _ptr_i32(n_free, "n_free"), int(B), int(B_out), int(num_pages), int(page_size),
                              int(max_pages_per_seq), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "fa_pages_fork")


def fa_pages_compact(pools, block_table, seqlens, block_table_out, n_live, B, num_pages, page_size,
                     max_pages_per_seq, workspace, workspace_bytes, stream=None) -> None:
    arr = _pool_array(pools, int(num_pages))
    st = load().fa_pages_compact(_pool_ptr(arr), len(pools), _ptr_i32(block_table, "block_table"),
                                 _ptr_i32(seqlens, "seqlens"), _ptr_i32(block_table_out, "block_table_out"),
                                 _ptr_i32(n_live, "n_live"), int(B), int(num_pages), int(page_size),
                                 int(max_pages_per_seq), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "fa_pages_compact")


def fa_pages_workspace_size(num_pages, B_out=0) -> int:
    return int(load().fa_pages_workspace_size(int(num_pages), int(B_out)))


def fa_selftest_wait_timeout(stream=None) -> None:
    """Launch the self-test whose bounded wait must run out (see include/fa.h)."""
    _check(load().fa_selftest_wait_timeout(_stream(stream)), "fa_selftest_wait_timeout")


def fa_last_device_error(stream=None) -> int:
    return int(load().fa_last_device_error(_stream(stream)))


def fa_device_sm_count() -> int:
    return int(load().fa_device_sm_count())


# ------------------------------------------------------------------ tensor-level helpers
# (a `stream` argument is a torch stream or a raw handle; a call with one runs as under torch.cuda.stream(stream))
def _other_stream(stream, t):
    """None, or the context of a launch on `stream` that is not torch's current stream of t's device:
    what the call allocates then belongs to `stream`, so that its memory is not given out again
    while kernels there use it."""
    import torch
    if not t.is_cuda:
        return None  # refused where its address is taken
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if handle == torch.cuda.current_stream(t.device).cuda_stream:
        return None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, t.device) if handle else torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream: expected one of {t.device}, got one of {stream.device}")
    return torch.cuda.stream(stream)


def _results_from(results):
    """Results that were allocated on another stream, for use on the current one too."""
    import torch
    for r in results:
        if r is not None:
            r.record_stream(torch.cuda.current_stream(r.device))
    return results


def forward(q, k, v, causal=False, scale=None, cu_seqlens=None, out=None, lse=None, workspace=None, stream=None,
            tf32=False):
    """O, lse for q [B,Nq,Hq,d] / k,v [B,Nk,Hkv,d] (or packed [total,H,d] with cu_seqlens).

    bf16 inputs give bf16 O; fp32 inputs (fixed length) are rounded to bf16 on the device and
    give fp32 O.  Outputs and workspace are allocated with torch unless passed in."""
    import torch
    varlen = cu_seqlens is not None
    _same("k, v", k, v)
    if q.dtype != k.dtype or q.shape[-1] != k.shape[-1] or q.dim() != k.dim():
        raise ValueError(f"q {q.dtype} {tuple(q.shape)} does not match k {k.dtype} {tuple(k.shape)}")
    if varlen:
        _require("q", q.dim() == 3, f"packed [total, Hq, d] with cu_seqlens, got shape {tuple(q.shape)}")
        total, Hq, d = q.shape
        Hkv = k.shape[1]
        _require("k", k.shape[0] == total, f"{total} packed rows like q, got {k.shape[0]}")
        _require("cu_seqlens", cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2,
                 f"[B + 1] offsets, got shape {tuple(cu_seqlens.shape)}")
        B, Nq, Nk = cu_seqlens.numel() - 1, total, total
        lse_shape = (Hq, total)
    else:
        _require("q", q.dim() == 4, f"[B, Nq, Hq, d], got shape {tuple(q.shape)}")
        B, Nq, Hq, d = q.shape
        Nk, Hkv = k.shape[1], k.shape[2]
        _require("k", k.shape[0] == B, f"batch {B} like q, got {k.shape[0]}")
        lse_shape = (B, Hq, Nq)
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    in_dtype = (FA_TF32 if tf32 else FA_F32) if q.dtype == torch.float32 else FA_BF16
    if scale is None:
        scale = d ** -0.5
    _expect(out, q.shape, "torch.bfloat16" if in_dtype == FA_BF16 else "torch.float32", "out")
    _expect(lse, lse_shape, "torch.float32", "lse")
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = forward(q, k, v, causal, scale, cu_seqlens, out, lse, workspace, None, tf32)
            return _results_from(done)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16 if in_dtype == FA_BF16 else torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    ws_bytes = fa_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, d, in_dtype, varlen)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    fa_fwd(q, k, v, out, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, cu_seqlens, in_dtype, workspace,
           ws_bytes if workspace is not None else 0, stream)
    return out, lse


def decode(q, kcache, vcache, seqlens=None, scale=None, split_len=1024, out=None, lse=None, workspace=None,
           stream=None):
    """O [B,Hq,d], lse [B,Hq] for one query token per sequence over caches [B,Lmax,Hkv,d]."""
    import torch
    _require("q", q.dim() == 3, f"[B, Hq, d], got shape {tuple(q.shape)}")
    B, Hq, d = q.shape
    _same("kcache, vcache", kcache, vcache)
    _bf16("decode", q, kcache)
    _require("kcache", kcache.dim() == 4 and kcache.shape[0] == B and kcache.shape[3] == d,
             f"[B={B}, Lmax, Hkv, d={d}], got shape {tuple(kcache.shape)}")
    Lmax, Hkv = kcache.shape[1], kcache.shape[2]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    _lengths(seqlens, B, "seqlens")
    if scale is None:
        scale = d ** -0.5
    _expect(out, (B, Hq, d), "torch.bfloat16", "out")
    _expect(lse, (B, Hq), "torch.float32", "lse")
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = decode(q, kcache, vcache, seqlens, scale, split_len, out, lse, workspace)
            return _results_from(done)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws_bytes = fa_decode_workspace_size(B, Hq, Lmax, d, split_len)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    fa_decode(q, kcache, vcache, seqlens, out, lse, B, Hq, Hkv, Lmax, d, scale, split_len, workspace, ws_bytes,
              stream)
    return out, lse


def decode_paged(q, k_pages, v_pages, block_table, seqlens, scale=None, split_len=1024, out=None, lse=None,
                 workspace=None, stream=None):
    """O [B,Hq,d], lse [B,Hq] for one query token per sequence over a page pool
    [num_pages, page_size, Hkv, d] addressed by block_table [B, max_pages] (int32) and
    seqlens [B] (int32)."""
    import torch
    _require("q", q.dim() == 3, f"[B, Hq, d], got shape {tuple(q.shape)}")
    B, Hq, d = q.shape
    _same("k_pages, v_pages", k_pages, v_pages)
    _bf16("decode_paged", q, k_pages)
    _require("k_pages", k_pages.dim() == 4 and k_pages.shape[3] == d,
             f"[num_pages, page_size, Hkv, d={d}], got shape {tuple(k_pages.shape)}")
    num_pages, page_size, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    _lengths(seqlens, B, "seqlens")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table: expected [B={B}, max_pages], got {tuple(block_table.shape)}")
    maxp = block_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    _expect(out, (B, Hq, d), "torch.bfloat16", "out")
    _expect(lse, (B, Hq), "torch.float32", "lse")
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, split_len, out, lse,
                                    workspace)
            return _results_from(done)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws_bytes = fa_decode_paged_workspace_size(B, Hq, Hkv, maxp, page_size, d, split_len)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    fa_decode_paged(q, k_pages, v_pages, block_table, seqlens, out, lse, B, Hq, Hkv, num_pages, page_size, maxp, d,
                    scale, split_len, workspace, ws_bytes, stream)
    return out, lse


def backward(q, k, v, o, lse, dout, causal=False, scale=None, workspace=None, stream=None):
    """dq, dk, dv for q [B,Nq,Hq,d], k/v [B,Nk,Hkv,d], the forward's o and lse, and dout."""
    import torch
    _require("q", q.dim() == 4, f"[B, Nq, Hq, d], got shape {tuple(q.shape)}")
    B, Nq, Hq, d = q.shape
    _same("q, o, dout", q, o, dout)
    _same("k, v", k, v)
    _bf16("backward", q, k)
    _require("k", k.dim() == 4 and k.shape[0] == B and k.shape[3] == d,
             f"[B={B}, Nk, Hkv, d={d}], got shape {tuple(k.shape)}")
    Nk, Hkv = k.shape[1], k.shape[2]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    _expect(lse, (B, Hq, Nq), "torch.float32", "lse")
    if scale is None:
        scale = d ** -0.5
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = backward(q, k, v, o, lse, dout, causal, scale, workspace)
            return _results_from(done)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws_bytes = fa_bwd_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, Nq, Nk, d, scale, causal, workspace, ws_bytes, stream)
    return dq, dk, dv


def backward_varlen(q, k, v, o, lse, dout, cu_seqlens, causal=False, scale=None, workspace=None, stream=None):
    """dq, dk, dv for packed sequences: q, o, dout [total,Hq,d], k/v [total,Hkv,d], lse [Hq,total]
    from the varlen forward, cu_seqlens int32 [B+1] on the device."""
    import torch
    _require("q", q.dim() == 3, f"packed [total, Hq, d], got shape {tuple(q.shape)}")
    total, Hq, d = q.shape
    _same("q, o, dout", q, o, dout)
    _same("k, v", k, v)
    _bf16("backward_varlen", q, k)
    _require("k", k.dim() == 3 and k.shape[0] == total and k.shape[2] == d,
             f"[total={total}, Hkv, d={d}], got shape {tuple(k.shape)}")
    _require("cu_seqlens", cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2,
             f"[B + 1] offsets, got shape {tuple(cu_seqlens.shape)}")
    Hkv = k.shape[1]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    B = cu_seqlens.numel() - 1
    _expect(lse, (Hq, total), "torch.float32", "lse")
    if scale is None:
        scale = d ** -0.5
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = backward_varlen(q, k, v, o, lse, dout, cu_seqlens, causal, scale, workspace)
            return _results_from(done)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws_bytes = fa_bwd_varlen_workspace_size(B, Hq, total, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, total, d, scale, causal, cu_seqlens, workspace,
                  ws_bytes, stream)
    return dq, dk, dv


def forward_qkvpacked(qkv, causal=False, scale=None, cu_seqlens=None):
    """O, lse for qkv [B,N,3,H,d] (or [total,3,H,d] with cu_seqlens), bf16."""
    import torch
    if cu_seqlens is not None:
        _require("qkv", qkv.dim() == 4 and qkv.shape[1] == 3, f"[total, 3, H, d], got shape {tuple(qkv.shape)}")
        total, _, H, d = qkv.shape
        B, N = cu_seqlens.numel() - 1, total
        out = torch.empty((total, H, d), dtype=torch.bfloat16, device=qkv.device)
        lse = torch.empty((H, total), dtype=torch.float32, device=qkv.device)
    else:
        _require("qkv", qkv.dim() == 5 and qkv.shape[2] == 3, f"[B, N, 3, H, d], got shape {tuple(qkv.shape)}")
        B, N, _, H, d = qkv.shape
        out = torch.empty((B, N, H, d), dtype=torch.bfloat16, device=qkv.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=qkv.device)
    if scale is None:
        scale = d ** -0.5
    fa_fwd_qkvpacked(qkv, out, lse, B, H, N, d, scale, causal, cu_seqlens)
    return out, lse


def forward_fp8(q8, k8, v8, descale_q, descale_k, descale_v, causal=False, scale=None, workspace=None):
    """O (bf16), lse for e4m3 q8 [B,Nq,Hq,128], k8/v8 [B,Nk,Hkv,128] (uint8 or float8 tensors)."""
    import torch
    _require("q8", q8.dim() == 4, f"[B, Nq, Hq, d], got shape {tuple(q8.shape)}")
    B, Nq, Hq, d = q8.shape
    _same("k8, v8", k8, v8)
    _require("k8", k8.dim() == 4 and k8.shape[0] == B and k8.shape[3] == d,
             f"[B={B}, Nk, Hkv, d={d}], got shape {tuple(k8.shape)}")
    Nk, Hkv = k8.shape[1], k8.shape[2]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    if scale is None:
        scale = d ** -0.5
    o = torch.empty((B, Nq, Hq, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q8.device)
    ws_bytes = fa_fwd_fp8_workspace_size(B, Hkv, Nk, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q8.device)
    fa_fwd_fp8(q8, k8, v8, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, descale_q, descale_k, descale_v, causal, workspace,
               ws_bytes)
    return o, lse


# ------------------------------------------------------------------ rotary positions, 8-bit cache, pages
def _home(first, *others) -> int:
    """Index of the device that holds every tensor (launches go to the current device, so the
    calls below make it current)."""
    idx = first.get_device()
    if idx < 0:
        raise ValueError(f"expected a CUDA tensor, got one on {first.device}")
    for t in others:
        if t is not None and t.get_device() != idx:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return idx


def _elsewhere(idx: int) -> bool:
    import torch
    return idx != torch.cuda.current_device()


def _dense(**tensors) -> None:
    for what, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous tensor, got strides {tuple(t.stride())} for shape "
                             f"{tuple(t.shape)}")


def _is_i32(**tensors) -> None:
    import torch
    for what, t in tensors.items():
        if t is not None and t.dtype != torch.int32:
            raise ValueError(f"{what}: expected an int32 tensor, got {t.dtype}")


_ROPE_SCALINGS = {"none": FA_ROPE_NONE, "linear": FA_ROPE_LINEAR, "ntk": FA_ROPE_NTK, "bands": FA_ROPE_BANDS}


def rope_frequencies(rot_dim, theta=10000.0, scaling="none", factor=1.0, original_len=0, low=1.0, high=32.0,
                     device="cuda"):
    """float64 [rot_dim / 2] angular frequencies on `device`, for rope(); made once and kept.
    scaling: "none", "linear", "ntk" or "bands" (see fa_rope_scaling in include/fa.h)."""
    import torch
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling: expected one of {sorted(_ROPE_SCALINGS)}, got {scaling!r}")
    return torch.tensor(fa_rope_frequencies(rot_dim, theta, _ROPE_SCALINGS[scaling], factor, original_len, low, high),
                        dtype=torch.float64, device=device)


def _row_stride(t, what: str) -> int:
    """Elements between rows of [..., H, d] whose heads are dense and whose rows are evenly
    spaced (a dense tensor, or q or k inside a packed [..., 3, H, d] one)."""
    H, d = t.shape[-2:]
    if t.is_contiguous():
        return H * d
    ok = t.stride(-1) == 1 and (H == 1 or t.stride(-2) == d)
    step = H * d
    lead = [(n, s) for n, s in zip(t.shape[:-2], t.stride()[:-2]) if n != 1]
    if lead:
        step = lead[-1][1]
        for (n0, s0), (n1, s1) in zip(lead, lead[1:]):
            ok = ok and s0 == n1 * s1
    if not ok or step < H * d:
        raise ValueError(f"{what}: expected dense heads and evenly spaced rows, got strides {tuple(t.stride())} for "
                         f"shape {tuple(t.shape)}")
    return step


def _rope(q, k, freqs, positions, interleaved, amplitude, q_out, k_out, stream, backward):
    import torch
    dt, qs = q.dtype, q.shape
    if len(qs) not in (3, 4) or (dt != torch.bfloat16 and dt != torch.float32):
        raise ValueError(f"q: expected bf16 or fp32 [B, N, Hq, d] or [total, Hq, d], got {dt} {tuple(qs)}")
    period, Hq, d = qs[-3:]
    rows = period if len(qs) == 3 else period * qs[0]
    Hk = 0
    if k is not None:
        ks = k.shape
        Hk = ks[-2] if len(ks) > 1 else 0
        if k.dtype != dt or ks != (*qs[:-2], Hk, d):
            raise ValueError(f"k: expected {dt} {tuple(qs[:-2])} + (Hkv, {d}) like q, got {k.dtype} {tuple(ks)}")
    elif k_out is not None:
        raise ValueError("k_out given without k")
    rot = 2 * freqs.numel()
    if freqs.dtype != torch.float64 or not 0 < rot <= d or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError(f"freqs: expected dense float64 [rot_dim / 2] with rot_dim <= {d}, got {freqs.dtype} "
                         f"{tuple(freqs.shape)}")
    if positions is not None:
        if positions.numel() != rows or (positions.dim() != 1 and positions.shape != qs[:-2]):
            raise ValueError(f"positions: expected {tuple(qs[:-2])} or [{rows}], got shape {tuple(positions.shape)}")
        if positions.dtype != torch.int32 or not positions.is_contiguous():
            raise ValueError(f"positions: expected a dense int32 tensor, got {positions.dtype}, strides "
                             f"{tuple(positions.stride())}")
    if q_out is not None and (q_out.shape != qs or q_out.dtype != dt):
        raise ValueError(f"q_out: expected {dt} {tuple(qs)}, got {q_out.dtype} {tuple(q_out.shape)}")
    if k_out is not None and (k_out.shape != ks or k_out.dtype != dt):
        raise ValueError(f"k_out: expected {dt} {tuple(ks)}, got {k_out.dtype} {tuple(k_out.shape)}")
    if _elsewhere(_home(q, k, freqs, positions, q_out, k_out)):
        with torch.cuda.device(q.device):
            return _rope(q, k, freqs, positions, interleaved, amplitude, q_out, k_out, stream, backward)
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = _rope(q, k, freqs, positions, interleaved, amplitude, q_out, k_out, None, backward)
            return _results_from(done)
    # like the input where that is dense; empty_like would keep the strides of a slice's dimensions
    dense = Hq * d
    sq = syq = dense
    if not q.is_contiguous():
        sq = _row_stride(q, "q")
    if q_out is None:
        q_out = torch.empty_like(q) if sq == dense else q.new_empty(qs)
    elif not q_out.is_contiguous():
        syq = _row_stride(q_out, "q_out")
    sk = syk = Hk * d
    if k is not None:
        if not k.is_contiguous():
            sk = _row_stride(k, "k")
        if k_out is None:
            k_out = torch.empty_like(k) if sk == Hk * d else k.new_empty(ks)
        elif not k_out.is_contiguous():
            syk = _row_stride(k_out, "k_out")
    if rows > 0:
        st = load().fa_rope(q.data_ptr(), k.data_ptr() if Hk else None, q_out.data_ptr(),
                            k_out.data_ptr() if Hk else None, None if positions is None else positions.data_ptr(),
                            freqs.data_ptr(), rows, period, Hq, Hk, d, rot, 1 if interleaved else 0, amplitude,
                            1 if backward else 0, FA_BF16 if dt == torch.bfloat16 else FA_F32, sq, sk, syq, syk,
                            _stream(stream))
        if st != FA_OK:
            raise FaError(st, "fa_rope")
    return q_out, k_out


def rope(q, k, freqs, positions=None, interleaved=False, amplitude=1.0, q_out=None, k_out=None, stream=None):
    """q and k (or None) turned by their positions: [B, N, H, d] or packed [total, H, d], bf16 or
    fp32; q and k may be slices of a packed qkv tensor.  freqs from rope_frequencies();
    positions int32, one per row, or None: 0 .. N - 1 (0 .. total - 1).  q_out / k_out may be q / k
    themselves.  Returns (q_out, k_out)."""
    return _rope(q, k, freqs, positions, interleaved, amplitude, q_out, k_out, stream, False)


def rope_backward(dq, dk, freqs, positions=None, interleaved=False, amplitude=1.0, q_out=None, k_out=None,
                  stream=None):
    """Gradients of rope()'s inputs from those of its outputs (same arguments as rope())."""
    return _rope(dq, dk, freqs, positions, interleaved, amplitude, q_out, k_out, stream, True)


def _cache8(k_pages, v_pages, k_scale, v_scale, block_table, seqlens):
    """Checks an e4m3 paged cache; returns (B, num_pages, page_size, max_pages, Hkv, d, scale_block)."""
    import torch
    shape, dt, ks = k_pages.shape, k_pages.dtype, k_scale.shape
    if shape != v_pages.shape or dt != v_pages.dtype or len(shape) != 4 or \
            (dt != torch.float8_e4m3fn and dt != torch.uint8):
        raise ValueError(f"k_pages, v_pages: expected two e4m3 (or byte) [num_pages, page_size, Hkv, d], got "
                         f"{dt} {tuple(shape)} and {v_pages.dtype} {tuple(v_pages.shape)}")
    num_pages, page_size, Hkv, d = shape
    if ks != v_scale.shape or len(ks) != 3 or ks[0] != num_pages or ks[1] != Hkv or ks[2] <= 0 or \
            page_size % ks[2] != 0 or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise ValueError(f"k_scale, v_scale: expected two float32 [{num_pages}, {Hkv}, page_size / scale_block], got "
                         f"{k_scale.dtype} {tuple(ks)} and {v_scale.dtype} {tuple(v_scale.shape)}")
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [B, max_pages], got {tuple(block_table.shape)}")
    B, maxp = block_table.shape
    if seqlens.dim() != 1 or seqlens.shape[0] != B:
        raise ValueError(f"seqlens: expected {B} entries, got shape {tuple(seqlens.shape)}")
    if block_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise ValueError(f"block_table, seqlens: expected int32 tensors, got {block_table.dtype} and {seqlens.dtype}")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous() and k_scale.is_contiguous() and
            v_scale.is_contiguous() and block_table.is_contiguous() and seqlens.is_contiguous()):
        raise ValueError("expected contiguous tensors: pages, scales, block_table, seqlens")
    return B, num_pages, page_size, maxp, Hkv, d, page_size // ks[2]


def cache_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, cu_seqlens=None, stream=None):
    """Writes bf16 k, v [total, Hkv, d] into an e4m3 paged cache (pages [num_pages, page_size, Hkv,
    d], scales float32 [num_pages, Hkv, page_size / scale_block]), in place.  seqlens [B]: lengths
    with the new rows; cu_seqlens [B + 1]: the new rows of each sequence, or None: one each."""
    import torch
    if k.shape != v.shape or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError(f"k, v: expected two bf16 tensors of one shape, got {k.dtype} {tuple(k.shape)} and {v.dtype} "
                         f"{tuple(v.shape)}")
    B, P, ps, maxp, Hkv, d, sb = _cache8(k_pages, v_pages, k_scale, v_scale, block_table, seqlens)
    if k.dim() != 3 or k.shape[1] != Hkv or k.shape[2] != d:
        raise ValueError(f"k: expected [total, Hkv={Hkv}, d={d}], got shape {tuple(k.shape)}")
    total = k.shape[0]
    if cu_seqlens is None:
        if total != B:
            raise ValueError(f"k: expected one row for each of {B} sequences without cu_seqlens, got {total}")
    elif cu_seqlens.dim() != 1 or cu_seqlens.shape[0] != B + 1:
        raise ValueError(f"cu_seqlens: expected [B + 1 = {B + 1}] offsets, got shape {tuple(cu_seqlens.shape)}")
    if _elsewhere(_home(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, cu_seqlens)):
        with torch.cuda.device(k.device):
            return cache_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, cu_seqlens, stream)
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError(f"k, v: expected contiguous tensors, got strides {tuple(k.stride())} and {tuple(v.stride())}")
    if cu_seqlens is not None:
        _is_i32(cu_seqlens=cu_seqlens)
        _dense(cu_seqlens=cu_seqlens)

    if B > 0 and total > 0:
        _check(load().fa_cache_append_fp8(k.data_ptr(), v.data_ptr(),
                                          None if cu_seqlens is None else cu_seqlens.data_ptr(),
                                          block_table.data_ptr(), seqlens.data_ptr(), k_pages.data_ptr(),
                                          v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), B, total, Hkv, P,
                                          ps, maxp, sb, d, _stream(stream)), "fa_cache_append_fp8")


def decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, scale=None, out=None, lse=None,
                     workspace=None, stream=None):
    """O, lse for the newest tokens of each sequence over an e4m3 paged cache (see
    cache_append_fp8): q [B, Hq, d] gives lse [B, Hq]; q [B, Nq, Hq, d] (the Nq newest tokens,
    causal among themselves) gives lse [B, Hq, Nq]."""
    import torch
    if q.dtype != torch.bfloat16:
        raise ValueError(f"decode_paged_fp8: expected bf16 tensors, got {q.dtype}")
    B, P, ps, maxp, Hkv, d, sb = _cache8(k_pages, v_pages, k_scale, v_scale, block_table, seqlens)
    shape = q.shape
    if q.dim() not in (3, 4) or shape[0] != B or shape[-1] != d:
        raise ValueError(f"q: expected [B={B}, Hq, d={d}] or [B={B}, Nq, Hq, d={d}], got shape {tuple(shape)}")
    Nq, Hq = (shape[1] if q.dim() == 4 else 1), shape[-2]
    _require("heads", Hkv > 0 and Hq % Hkv == 0, f"Hq ({Hq}) a multiple of Hkv ({Hkv})")
    lse_shape = (B, Hq) if q.dim() == 3 else (B, Hq, Nq)
    if scale is None:
        scale = d ** -0.5
    if out is not None:
        _expect(out, shape, "torch.bfloat16", "out")
    if lse is not None:
        _expect(lse, lse_shape, "torch.float32", "lse")
    if _elsewhere(_home(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, out, lse, workspace)):
        with torch.cuda.device(q.device):
            return decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, scale, out, lse,
                                    workspace, stream)
    if stream is not None:
        other = _other_stream(stream, q)
        if other:
            with other:
                done = decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, scale, out, lse,
                                        workspace)
            return _results_from(done)
    if not q.is_contiguous():
        raise ValueError(f"q: expected a contiguous tensor, got strides {tuple(q.stride())} for shape {tuple(shape)}")
    if out is not None or lse is not None or workspace is not None:
        _dense(out=out, lse=lse, workspace=workspace)

    lib = load()
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = q.new_empty(lse_shape, dtype=torch.float32)
    if workspace is None:
        nbytes = lib.fa_decode_paged_fp8_workspace_size(B, Nq, Hq, Hkv, d)
        workspace = q.new_empty(max(nbytes, 1), dtype=torch.uint8)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    if B > 0 and Nq > 0 and Hq > 0:
        _check(lib.fa_decode_paged_fp8(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                                       v_scale.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                       lse.data_ptr(), B, Nq, Hq, Hkv, P, ps, maxp, sb, d, scale,
                                       workspace.data_ptr(), nbytes, _stream(stream)), "fa_decode_paged_fp8")
    return out, lse


def _paged_table(pools, block_table, seqlens, num_pages):
    """Checks the table of a paged cache of any element type; returns (B, max_pages, num_pages)."""
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [B, max_pages], got {tuple(block_table.shape)}")
    B, maxp = block_table.shape
    if seqlens.dim() != 1 or seqlens.shape[0] != B:
        raise ValueError(f"seqlens: expected {B} entries, got shape {tuple(seqlens.shape)}")
    if num_pages is None:
        if not len(pools):
            raise ValueError("pools: expected at least one pool, or num_pages")
        num_pages = pools[0].shape[0]
    _is_i32(block_table=block_table, seqlens=seqlens)
    _dense(block_table=block_table, seqlens=seqlens)
    return B, maxp, num_pages


def pages_fork(pools, block_table, seqlens, parent, page_size, num_pages=None, workspace=None, stream=None):
    """Sequence i of the result continues sequence parent[i] (int32; -1: empty).  Full pages are
    shared, a partly filled last page is copied for all but one of its heirs in every pool (a list
    of tensors [num_pages, ...]).  Returns (block_table, seqlens, free_pages [num_pages], n_free
    [1]); see fa_pages_fork in include/fa.h."""
    import torch
    B, maxp, num_pages = _paged_table(pools, block_table, seqlens, num_pages)
    if parent.dim() != 1:
        raise ValueError(f"parent: expected [B_out], got shape {tuple(parent.shape)}")
    R = parent.shape[0]
    _is_i32(parent=parent)
    _dense(parent=parent, workspace=workspace)

    if _elsewhere(_home(block_table, seqlens, parent, workspace, *pools)):
        with torch.cuda.device(block_table.device):
            return pages_fork(pools, block_table, seqlens, parent, page_size, num_pages, workspace, stream)
    if stream is not None:
        other = _other_stream(stream, block_table)
        if other:
            with other:
                done = pages_fork(pools, block_table, seqlens, parent, page_size, num_pages, workspace)
            return _results_from(done)
    lib = load()
    arr = _pool_array(pools, num_pages)
    # one allocation for the four results
    buf = block_table.new_empty(R * (maxp + 1) + num_pages + 1)
    table, lens, free, n_free = buf.split((R * maxp, R, num_pages, 1))
    if workspace is None:
        nbytes = lib.fa_pages_workspace_size(num_pages, R)
        workspace = block_table.new_empty(max(nbytes, 1), dtype=torch.uint8)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(lib.fa_pages_fork(_pool_ptr(arr), len(pools), block_table.data_ptr(), seqlens.data_ptr(), parent.data_ptr(),
                             table.data_ptr(), lens.data_ptr(), free.data_ptr(), n_free.data_ptr(), B, R, num_pages,
                             page_size, maxp, workspace.data_ptr(), nbytes, _stream(stream)), "fa_pages_fork")
    return table.view(R, maxp), lens, free, n_free


def pages_compact(pools, block_table, seqlens, page_size, num_pages=None, workspace=None, stream=None):
    """Moves the pages in use to the front of every pool.  Returns (block_table, n_live [1])."""
    import torch
    B, maxp, num_pages = _paged_table(pools, block_table, seqlens, num_pages)
    _dense(workspace=workspace)

    if _elsewhere(_home(block_table, seqlens, workspace, *pools)):
        with torch.cuda.device(block_table.device):
            return pages_compact(pools, block_table, seqlens, page_size, num_pages, workspace, stream)
    if stream is not None:
        other = _other_stream(stream, block_table)
        if other:
            with other:
                done = pages_compact(pools, block_table, seqlens, page_size, num_pages, workspace)
            return _results_from(done)
    lib = load()
    arr = _pool_array(pools, num_pages)
    table, n_live = torch.empty_like(block_table), block_table.new_empty(1)
    if workspace is None:
        nbytes = lib.fa_pages_workspace_size(num_pages, 0)
        workspace = block_table.new_empty(max(nbytes, 1), dtype=torch.uint8)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _check(lib.fa_pages_compact(_pool_ptr(arr), len(pools), block_table.data_ptr(), seqlens.data_ptr(), table.data_ptr(),
                                n_live.data_ptr(), B, num_pages, page_size, maxp, workspace.data_ptr(), nbytes,
                                _stream(stream)), "fa_pages_compact")
    return table, n_live

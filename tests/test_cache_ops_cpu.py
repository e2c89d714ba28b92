"""CPU-side checks of the rotary, 8-bit cache and page operators: the C ABI and the binding refuse
bad arguments before anything is launched, and the frequencies are the formulas'."""
import ctypes
import math

import pytest
import torch

from exact_io_aware_97_b200 import binding as fa
from exact_io_aware_97_b200 import build as fa_build


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load()


BAD, UNS, WS, OK = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE, fa.FA_OK


def test_rope_rejects_before_launch(lib):
    def st(**kw):
        a = dict(q=256, k=512, qo=256, ko=512, pos=None, f=1024, rows=4, period=4, Hq=2, Hk=1, d=64, rot=64, inter=0,
                 amp=1.0, back=0, dt=0, qs=128, ks=64, qos=128, kos=64)
        a.update(kw)
        return lib.fa_rope(a["q"], a["k"], a["qo"], a["ko"], a["pos"], a["f"], a["rows"], a["period"], a["Hq"],
                           a["Hk"], a["d"], a["rot"], a["inter"], ctypes.c_float(a["amp"]), a["back"], a["dt"],
                           a["qs"], a["ks"], a["qos"], a["kos"], None)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(f=None), dict(f=1028), dict(pos=513),
               dict(period=0), dict(rot=0), dict(rot=63), dict(rot=66), dict(rows=-1), dict(Hq=0), dict(Hk=-1),
               dict(dt=2), dict(dt=9), dict(amp=math.inf), dict(q=264), dict(ko=520), dict(qs=127), dict(qs=120),
               dict(ks=68), dict(qos=256), dict(kos=72)):
        assert st(**kw) == BAD, kw
    for kw in (dict(d=96), dict(rows=1 << 31), dict(Hq=65535, qs=65535 * 64, qos=65535 * 64)):
        assert st(**kw) == UNS, kw
    assert st(rows=0) == OK


def test_rope_frequencies_are_the_formulas(lib):
    for rot, theta in ((2, 10000.0), (64, 10000.0), (128, 500000.0)):
        plain = [theta ** (-2 * i / rot) for i in range(rot // 2)]
        close = lambda a, b: all(abs(x - y) <= 1e-13 * y for x, y in zip(a, b, strict=True))  # noqa: E731
        assert close(fa.fa_rope_frequencies(rot, theta), plain)
        assert close(fa.fa_rope_frequencies(rot, theta, fa.FA_ROPE_LINEAR, 4.0), [w / 4 for w in plain])
        t2 = theta * 4.0 ** (rot / (rot - 2)) if rot > 2 else theta
        assert close(fa.fa_rope_frequencies(rot, theta, fa.FA_ROPE_NTK, 4.0),
                     [t2 ** (-2 * i / rot) for i in range(rot // 2)])
        bands = []
        for w in plain:
            keep = min(1.0, max(0.0, (4096 * w / (2 * math.pi) - 1) / 31))
            bands.append(w * (keep + (1 - keep) / 8))
        assert close(fa.fa_rope_frequencies(rot, theta, fa.FA_ROPE_BANDS, 8.0, 4096, 1.0, 32.0), bands)
    for bad in ((0,), (-2,), (7,), (8, 0.0), (8, math.nan), (8, 1e4, 5), (8, 1e4, fa.FA_ROPE_LINEAR, 0.0),
                (8, 1e4, fa.FA_ROPE_BANDS, 2.0, 0.0, 1.0, 2.0), (8, 1e4, fa.FA_ROPE_BANDS, 2.0, 4096, 3.0, 3.0)):
        with pytest.raises(fa.FaError):
            fa.fa_rope_frequencies(*bad)
    with pytest.raises(ValueError, match="scaling"):
        fa.rope_frequencies(8, scaling="dynamic", device="cpu")


def _append(lib, **kw):
    a = dict(k=256, v=256, cu=None, bt=512, sl=512, kp=256, vp=256, ks=512, vs=512, B=2, total=2, Hkv=2, P=10, ps=32,
             maxp=4, sb=16, d=64)
    a.update(kw)
    return lib.fa_cache_append_fp8(*(a[n] for n in ("k", "v", "cu", "bt", "sl", "kp", "vp", "ks", "vs", "B", "total",
                                                    "Hkv", "P", "ps", "maxp", "sb", "d")), None)


def _decode(lib, **kw):
    a = dict(q=256, kp=256, vp=256, ks=512, vs=512, bt=512, sl=512, o=256, lse=None, B=2, Nq=1, Hq=4, Hkv=2, P=10,
             ps=32, maxp=4, sb=16, d=64, scale=0.1, ws=256, wsb=1 << 30)
    a.update(kw)
    return lib.fa_decode_paged_fp8(*(a[n] for n in ("q", "kp", "vp", "ks", "vs", "bt", "sl", "o", "lse", "B", "Nq",
                                                    "Hq", "Hkv", "P", "ps", "maxp", "sb", "d")),
                                   ctypes.c_float(a["scale"]), a["ws"], a["wsb"], None)


def test_cache8_rejects_before_launch(lib):
    for st in (_append, _decode):
        for kw in (dict(kp=None), dict(vp=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(sl=None),
                   dict(kp=264), dict(vp=8), dict(ks=514), dict(bt=513), dict(sl=514), dict(B=-1), dict(Hkv=0),
                   dict(P=0), dict(ps=0), dict(maxp=0), dict(sb=0)):
            assert st(lib, **kw) == BAD, kw
        for kw in (dict(ps=24), dict(ps=8, sb=8), dict(sb=8), dict(sb=24), dict(sb=64), dict(ps=512, sb=512),
                   dict(d=96), dict(P=1 << 26, ps=32), dict(maxp=1 << 26), dict(B=65536, total=65536),
                   dict(Hkv=65536, Hq=65536)):
            if st is _append:
                kw.pop("Hq", None)
            assert st(lib, **kw) == UNS, kw
    for kw in (dict(k=None), dict(v=None), dict(k=264), dict(total=-1), dict(total=3), dict(cu=514)):
        assert _append(lib, **kw) == BAD, kw
    assert _append(lib, B=0, total=0) == OK and _append(lib, cu=512, total=0) == OK
    for kw in (dict(q=None), dict(o=None), dict(q=264), dict(o=8), dict(lse=514), dict(Nq=-1), dict(Hq=0),
               dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf)):
        assert _decode(lib, **kw) == BAD, kw
    assert _decode(lib, Hq=3) == UNS
    for kw in (dict(ws=None), dict(wsb=0), dict(ws=264)):
        assert _decode(lib, **kw) == WS, kw
    assert _decode(lib, B=0) == OK and _decode(lib, Nq=0) == OK
    assert fa.fa_decode_paged_fp8_workspace_size(0, 1, 8, 8, 64) == 0


def test_pages_reject_before_launch(lib):
    def pools(*pairs):
        arr = (fa.FaPool * max(1, len(pairs)))()
        for n, (b, s) in enumerate(pairs):
            arr[n].base, arr[n].page_bytes = b, s
        return ctypes.cast(arr, ctypes.c_void_p)

    def fork(**kw):
        a = dict(p=pools((256, 64)), n=1, bt=512, sl=512, par=512, bto=1024, slo=1024, f=512, nf=512, B=2, R=2, P=10,
                 ps=16, maxp=4, ws=256, wsb=1 << 30)
        a.update(kw)
        return lib.fa_pages_fork(*(a[n] for n in ("p", "n", "bt", "sl", "par", "bto", "slo", "f", "nf", "B", "R", "P",
                                                  "ps", "maxp", "ws", "wsb")), None)

    def compact(**kw):
        a = dict(p=pools((256, 64)), n=1, bt=512, sl=512, bto=1024, nl=512, B=2, P=10, ps=16, maxp=4, ws=256,
                 wsb=1 << 30)
        a.update(kw)
        return lib.fa_pages_compact(*(a[n] for n in ("p", "n", "bt", "sl", "bto", "nl", "B", "P", "ps", "maxp", "ws",
                                                     "wsb")), None)
    for st in (fork, compact):
        for kw in (dict(n=-1), dict(p=None), dict(p=pools((None, 64))), dict(p=pools((256, 0))), dict(bt=None),
                   dict(sl=None), dict(bt=514), dict(sl=513), dict(bto=None), dict(bto=1026), dict(bto=512),
                   dict(B=-1), dict(P=0), dict(ps=0), dict(maxp=0)):
            assert st(**kw) == BAD, kw
        for kw in (dict(ps=24), dict(maxp=1 << 28), dict(P=0x7FFFFFFF), dict(p=pools((256, 1 << 31))), dict(n=4097, p=pools(*[(256, 16)] * 4097))):
            assert st(**kw) == UNS, kw
        for kw in (dict(ws=None), dict(wsb=100), dict(ws=260)):
            assert st(**kw) == WS, kw
    for kw in (dict(par=None), dict(slo=None), dict(slo=512), dict(f=None), dict(nf=None), dict(nf=514), dict(R=-1)):
        assert fork(**kw) == BAD, kw
    for kw in (dict(nl=None), dict(nl=513)):
        assert compact(**kw) == BAD, kw
    assert fa.fa_pages_workspace_size(0, 4) == 0
    assert fa.fa_pages_workspace_size(1000, 3000) >= 4 * (1000 + 3 * 3000)


def test_binding_refuses_before_the_library(lib):
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    q, k = torch.zeros(2, 5, 4, 64, dtype=bf), torch.zeros(2, 5, 2, 64, dtype=bf)
    freqs = fa.rope_frequencies(64, device="cpu")
    for match, args, kw in (("CUDA", (q, k, freqs), {}), ("freqs", (q, k, freqs.float()), {}),
                            ("freqs", (q, k, torch.zeros(33, dtype=torch.float64)), {}),
                            ("k:", (q, k[:1], freqs), {}), ("k:", (q, k.float(), freqs), {}),
                            ("q:", (q.half(), None, freqs), {}), ("positions", (q, k, freqs, torch.zeros(3, dtype=i32)), {}),
                            ("q_out", (q, k, freqs), dict(q_out=q[:1])), ("k_out", (q, None, freqs), dict(k_out=k))):
        for f in (fa.rope, fa.rope_backward):
            with pytest.raises(ValueError, match=match):
                f(*args, stream=0, **kw)
    with pytest.raises(ValueError, match="strides"):
        fa._row_stride(q.transpose(1, 2), "q")
    with pytest.raises(ValueError, match="strides"):
        fa._row_stride(torch.zeros(5, 4, 128, dtype=bf)[..., :64], "q")
    assert fa._row_stride(torch.zeros(2, 5, 3, 4, 64)[:, :, 1], "q") == 3 * 4 * 64

    kp = torch.zeros(6, 32, 2, 64, dtype=torch.uint8)
    ks = torch.zeros(6, 2, 2, dtype=f32)
    bt, sl = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    x = torch.zeros(3, 2, 64, dtype=bf)
    good = [x, x, kp, kp, ks, ks, bt, sl]
    for at, bad, match in ((0, x[:2], "k, v"), (2, kp.float(), "pages"), (3, kp[:5], "pages"), (4, ks[:, :1], "k_scale"),
                           (7, sl[:2], "seqlens"), (6, bt[0], "block_table"), (0, x.float(), "k, v")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            fa.cache_append_fp8(*args, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append_fp8(*good, stream=0)
    with pytest.raises(ValueError, match="bf16"):
        fa.cache_append_fp8(x.float(), x.float(), *good[2:], stream=0)
    with pytest.raises(ValueError, match="k:"):
        fa.cache_append_fp8(x[:2], x[:2], *good[2:], stream=0)
    with pytest.raises(ValueError, match="cu_seqlens"):
        fa.cache_append_fp8(*good, cu_seqlens=torch.zeros(3, dtype=i32), stream=0)
    with pytest.raises(ValueError, match="k_scale"):
        fa.cache_append_fp8(x, x, kp, kp, ks[:5], ks[:5], bt, sl, stream=0)
    qd = torch.zeros(3, 4, 64, dtype=bf)
    for match, args in (("q:", (qd[:2], kp, kp, ks, ks, bt, sl)), ("bf16", (qd.float(), kp, kp, ks, ks, bt, sl)),
                        ("heads", (qd[:, :3], kp, kp, ks, ks, bt, sl)), ("CUDA", (qd, kp, kp, ks, ks, bt, sl)),
                        ("q:", (qd[..., :32], kp, kp, ks, ks, bt, sl))):
        with pytest.raises(ValueError, match=match):
            fa.decode_paged_fp8(*args, stream=0)
    with pytest.raises(ValueError, match="out"):
        fa.decode_paged_fp8(qd, kp, kp, ks, ks, bt, sl, out=qd.float(), stream=0)
    with pytest.raises(ValueError, match="lse"):
        fa.decode_paged_fp8(qd, kp, kp, ks, ks, bt, sl, lse=torch.zeros(3, 4, 1), stream=0)
    for f in (lambda *a, **k: fa.pages_fork(a[0], a[1], a[2], sl, 32, **k),
              lambda *a, **k: fa.pages_compact(a[0], a[1], a[2], 32, **k)):
        for match, args in (("pools", ([], bt, sl)), ("block_table", ([kp], bt[0], sl)), ("seqlens", ([kp], bt, sl[:1])),
                            ("CUDA", ([kp], bt, sl))):
            with pytest.raises(ValueError, match=match):
                f(*args, stream=0)
    with pytest.raises(ValueError, match="pool 1"):
        fa._pool_array([(256, 4), kp[:3]], 6)

"""Calls with `stream=` other than torch's current stream: what they allocate belongs to that stream, and
calls on several streams at once, without workspaces of their own, give the results that one stream
gives."""
import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


class Spy:
    """The library, noting the addresses that the named functions get."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name.endswith("_size") or name in ("fa_last_device_error", "fa_status_string"):
            return f

        def call(*args):
            self.seen.append([a for a in args if isinstance(a, int) and a > 1 << 32])
            return f(*args)
        return call


def _owner(address):
    """Stream that the caching allocator keeps a device address for, or None."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


def _inputs():
    rng = np.random.default_rng(6401)
    lens, H, d, ps, sb = [1500, 70, 333], 2, 128, 32, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, extra=8)
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    q = torch.from_numpy(rng.standard_normal((3, 3, 16, d))).cuda().bfloat16()
    cache = (dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
    pools = [dev[0], dev[1], dev[2], dev[3]]
    parent = torch.tensor([2, 0, 0, 1], dtype=torch.int32, device="cuda")
    freqs = fa.rope_frequencies(d)
    return {
        "decode_paged_fp8": lambda stream=None: fa.decode_paged_fp8(q, *cache, stream=stream),
        "pages_fork": lambda stream=None: fa.pages_fork(pools, dev[4], dev[5], parent, ps, stream=stream),
        "pages_compact": lambda stream=None: fa.pages_compact([], dev[4], dev[5], ps, num_pages=kc.shape[0],
                                                              stream=stream),
        "rope": lambda stream=None: fa.rope(q, None, freqs, stream=stream)[:1],
        "rope_backward": lambda stream=None: fa.rope_backward(q, None, freqs, stream=stream)[:1],
        **_attention(),
    }


def _attention():
    g = torch.Generator(device="cuda").manual_seed(6402)
    q, k, v, dout = (torch.randn(2, 200, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    o, lse = fa.forward(q, k, v, causal=True)
    ov, lv = fa.forward(q[0], k[0], v[0], causal=True, cu_seqlens=cu)
    lens = torch.tensor([200, 77], dtype=torch.int32, device="cuda")
    pool = [x.reshape(-1, 16, 2, 64)[:24].contiguous() for x in (k, v)]
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12)
    plens = torch.tensor([190, 5], dtype=torch.int32, device="cuda")
    q32, k32, v32 = (x.float() for x in (q, k, v))
    q1 = q[:, 0].contiguous()
    return {
        "forward": lambda stream=None: fa.forward(q32, k32, v32, causal=True, stream=stream),
        "backward": lambda stream=None: fa.backward(q, k, v, o, lse, dout, causal=True, stream=stream)[1:],
        "backward_varlen": lambda stream=None: fa.backward_varlen(q[0], k[0], v[0], ov, lv, dout[0], cu, causal=True,
                                                                  stream=stream)[1:],
        "decode": lambda stream=None: fa.decode(q1, k, v, lens, split_len=64, stream=stream),
        "decode_paged": lambda stream=None: fa.decode_paged(q1, *pool, table, plens, split_len=64, stream=stream),
    }


@pytest.mark.parametrize("what", ["decode_paged_fp8", "pages_fork", "pages_compact", "rope", "rope_backward", "forward",
                                  "backward", "backward_varlen", "decode", "decode_paged"])
@pytest.mark.parametrize("form", ["stream", "handle"])
def test_memory_belongs_to_the_stream_of_the_call(what, form, monkeypatch):
    call = _inputs()[what]
    want = call()
    torch.cuda.synchronize()
    # (freed memory of the current stream that a call could be given)
    spare = [torch.empty(1 << k, dtype=torch.uint8, device="cuda") for k in range(10, 24)]
    del spare
    s = torch.cuda.Stream()
    known = {seg["address"]: seg for seg in torch.cuda.memory_snapshot()}
    spy = Spy(fa.load())
    monkeypatch.setattr(fa, "load", lambda *a: spy)
    got = call(s if form == "stream" else s.cuda_stream)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        assert _owner(a.data_ptr()) == s.cuda_stream
    # every address that the library got lies in the inputs' memory or in the call's stream's
    inputs_only = {address for address, seg in known.items() if seg["stream"] != s.cuda_stream}
    results = {a.data_ptr() for a in got}
    for address in spy.seen[-1]:
        if address == s.cuda_stream or address in results or _owner(address) is None:
            continue
        if _owner(address) != s.cuda_stream:
            blocks = [b for seg in torch.cuda.memory_snapshot() if seg["address"] in inputs_only for b in seg["blocks"]
                      if b["address"] <= address < b["address"] + b["size"]]
            assert blocks and blocks[0]["state"] == "active_allocated", hex(address)  # an input, still held


def test_calls_on_two_streams_while_the_current_one_allocates():
    calls = _inputs()
    want = {n: [t.clone() for t in c()] for n, c in calls.items() if n != "pages_fork"}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(40):
        for n, s in zip(("decode_paged_fp8", "pages_compact", "rope"), (streams[turn % 2], streams[1 - turn % 2],
                                                                        streams[turn % 2])):
            got.append((n, calls[n](s)))
            for size in (1 << 12, 1 << 16, 1 << 20, 1 << 22):  # what a freed workspace could be given to
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    for n, result in got:
        for a, b in zip(result, want[n]):
            assert torch.equal(a, b), n
    assert fa.fa_last_device_error() == fa.FA_OK


def test_the_current_stream_by_its_handle_and_the_default_one():
    calls = _inputs()
    want = calls["decode_paged_fp8"]()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for stream in (s, s.cuda_stream):
            o, lse = calls["decode_paged_fp8"](stream)
            assert _owner(o.data_ptr()) == s.cuda_stream
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        s.synchronize()
        o, lse = calls["decode_paged_fp8"](0)  # the legacy default stream
        assert _owner(o.data_ptr()) == 0
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_the_current_stream_without_torchs_raw_handle(monkeypatch):
    """The function that gives it is not a public one: where torch has none, calls find the stream."""
    calls = _inputs()
    want = calls["decode_paged_fp8"]()
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert fa._stream(None) == s.cuda_stream
    s.wait_stream(torch.cuda.current_stream())
    for n in ("rope", "decode_paged_fp8"):
        with torch.cuda.stream(s):
            got = calls[n]()
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

"""Rotary positions (fa_rope) against the pair formula in 64 bits, forward and gradient.

Tolerance: one rounding to the output type (half a step, 2^-8 of the value for bf16, 2^-24 for
fp32) plus the fp32 arithmetic before it.  The reduced angle (at most half a turn) is rounded to
fp32 once, sine and cosine are good to a few 2^-24, and each output is two products and a sum:
under 8 * 2^-24 of amplitude * (|x_a| + |x_b|)."""
import numpy as np
import pytest
import torch

import synth_inputs as si
from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


def turn64(x, pos, w, rot, interleaved, amplitude, back):
    """x float64 [rows, H, d]; returns (y, bound on |x_a| + |x_b| per element)."""
    a = np.outer(pos.astype(np.float64), w)
    c, s = amplitude * np.cos(a)[:, None], amplitude * np.sin(a)[:, None] * (-1 if back else 1)
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, m = x.copy(), np.zeros_like(x)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    m[..., ia] = m[..., ib] = amplitude * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return y, m


def check(y, x, pos, w, rot, interleaved, amplitude, back):
    d = x.shape[-1]
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    x64 = x.detach().double().cpu().numpy().reshape(-1, x.shape[-2], d)
    ref, m = turn64(x64, pos.reshape(-1), w, rot, interleaved, amplitude, back)
    got = y.double().cpu().numpy().reshape(ref.shape)
    assert np.array_equal(got[..., rot:], x64[..., rot:])  # the rest of the head is copied
    assert np.all(np.abs(got - ref) <= half * np.abs(ref) + 8 * 2.0 ** -24 * m)


def tensor(seed, tid, shape, dtype):
    x = si.normal(seed, tid, shape, "f32")
    return torch.from_numpy(x).cuda().to(dtype)


CASES = [
    # shape of q without heads, Hq, Hkv, d, rot, interleaved, dtype, first position
    ((1, 1), 64, 8, 128, 128, False, torch.bfloat16, 2000000),
    ((3, 5), 12, 12, 64, 64, True, torch.bfloat16, 0),
    ((2, 129), 8, 1, 128, 64, False, torch.bfloat16, 131071),
    ((77,), 4, 4, 64, 16, True, torch.float32, 9),
    ((2, 300), 6, 2, 128, 128, False, torch.float32, 4000000),
    ((33,), 3, 1, 64, 38, False, torch.bfloat16, 100),     # pairs that do not fill vectors
    ((33,), 3, 1, 128, 74, True, torch.bfloat16, 100),
    ((5,), 7, 1, 128, 2, False, torch.float32, 7),
    ((5,), 1, 3, 64, 2, True, torch.bfloat16, -50),        # negative positions turn backwards
    ((1, 2500), 16, 2, 128, 32, False, torch.bfloat16, 0),
]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}_{c[1]}_{c[2]}_d{c[3]}_r{c[4]}" for c in CASES])
def test_rope_matches_formula(case, back):
    lead, Hq, Hkv, d, rot, inter, dt, first = case
    q, k = tensor(4001, si.Q, (*lead, Hq, d), dt), tensor(4001, si.K, (*lead, Hkv, d), dt)
    freqs = fa.rope_frequencies(rot, 10000.0, "bands", 4.0, original_len=4096, low=1.0, high=32.0)
    pos = first + np.arange(int(np.prod(lead)))
    pt = torch.from_numpy(pos.astype(np.int32)).cuda().view(*lead)
    f = fa.rope_backward if back else fa.rope
    q0, k0 = q.clone(), k.clone()
    yq, yk = f(q, k, freqs, pt, interleaved=inter, amplitude=1.25)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    w = freqs.cpu().numpy()
    check(yq, q, pos, w, rot, inter, 1.25, back)
    check(yk, k, pos, w, rot, inter, 1.25, back)
    # in place, and q alone, give the same bits
    out = f(q, k, freqs, pt, interleaved=inter, amplitude=1.25, q_out=q, k_out=k)
    assert out[0] is q and torch.equal(q, yq) and torch.equal(k, yk)
    alone, none = f(q0, None, freqs, pt, interleaved=inter, amplitude=1.25)
    assert none is None and torch.equal(alone, yq)


def test_rope_default_positions_restart_with_each_sequence():
    q, k = tensor(4002, si.Q, (3, 7, 4, 64), torch.bfloat16), tensor(4002, si.K, (3, 7, 2, 64), torch.bfloat16)
    freqs = fa.rope_frequencies(64)
    yq, yk = fa.rope(q, k, freqs)
    pos = np.tile(np.arange(7), 3)
    check(yq, q, pos, freqs.cpu().numpy(), 64, False, 1.0, False)
    check(yk, k, pos, freqs.cpu().numpy(), 64, False, 1.0, False)
    assert torch.equal(yq[:, 0], q[:, 0])  # position 0


def test_rope_slices_of_a_packed_tensor():
    """q and k inside [B, N, 3, H, d], turned in place: v is not touched."""
    qkv = tensor(4003, si.Q, (2, 65, 3, 6, 128), torch.bfloat16)
    before = qkv.clone()
    freqs = fa.rope_frequencies(128)
    fa.rope(qkv[:, :, 0], qkv[:, :, 1], freqs, q_out=qkv[:, :, 0], k_out=qkv[:, :, 1])
    pos = np.tile(np.arange(65), 2)
    for j in (0, 1):
        check(qkv[:, :, j], before[:, :, j], pos, freqs.cpu().numpy(), 128, False, 1.0, False)
    assert torch.equal(qkv[:, :, 2], before[:, :, 2])


def test_rope_non_finite_stays_in_its_pair():
    q = tensor(4004, si.Q, (4, 2, 64), torch.bfloat16)
    q[1, 0, 3], q[2, 1, 40] = float("inf"), float("nan")
    freqs = fa.rope_frequencies(32)
    y, _ = fa.rope(q, None, freqs)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 19] = True  # columns 3 and 3 + 16 turn together
    want[2, 1, 40] = True                  # past the turned columns: copied
    assert torch.equal(bad, want)


def test_rope_gradient_against_differences():
    """<dy, rope(x + h u) - rope(x - h u)> / 2h = <rope_backward(dy), u> (linear: any h)."""
    x, u, dy = (tensor(4005, t, (11, 3, 64), torch.float32) for t in (1, 2, 3))
    freqs = fa.rope_frequencies(48, 500.0, "ntk", 2.0)
    pos = torch.arange(100, 111, dtype=torch.int32, device="cuda")
    f = lambda z: fa.rope(z, None, freqs, pos, interleaved=True, amplitude=0.75)[0].double()  # noqa: E731
    left = (dy.double() * (f(x + u) - f(x - u))).sum() / 2
    dx = fa.rope_backward(dy, None, freqs, pos, interleaved=True, amplitude=0.75)[0]
    right = (dx.double() * u.double()).sum()
    # each term carries a few 2^-24 of |dy| (|x| + |u|) or |dx| |u|
    scale = (dy.abs().double() * (x.abs() + u.abs()).double()).sum() + (dx.abs() * u.abs()).double().sum()
    assert abs(left - right) <= 16 * 2.0 ** -24 * scale


def test_rope_scores_depend_on_distance_only():
    """The attention around it: the same q and k shifted by 100000 positions give the same output
    up to the roundings of q, k (2^-8 each) and of the forward."""
    B, N, H, d = 1, 130, 2, 64
    q, k, v = (tensor(4006, t, (B, N, H, d), torch.bfloat16) for t in (1, 2, 3))
    freqs = fa.rope_frequencies(d)
    outs = []
    for first in (0, 100000):
        pos = first + torch.arange(N, dtype=torch.int32, device="cuda")
        o, _ = fa.forward(*fa.rope(q, k, freqs, pos), v, causal=True)
        outs.append(o.float())
    # scores are O(1) sums of 64 products, each within 2^-7 relative: their error is about
    # 2^-7 * |q||k| scale <= 2^-7 * 4 and that of o at most twice that times max|v| ~ 4
    assert (outs[0] - outs[1]).abs().max() <= 2 * 4 * 4 * 2.0 ** -7


def test_rope_in_training():
    """Forward and backward through rope and attention, against the oracle's backward on q and k
    turned in 64 bits, turned back in 64 bits.  Bounds of check_grad: rounding q and k after the
    turn adds one bf16 rounding (2^-8) to each element, of the size of those it already allows for."""
    import oracle as oracle_mod
    from parity import check_grad, host64
    orc = oracle_mod.get()
    B, N, Hq, H, d, rot = 1, 200, 4, 2, 64, 48
    q, dy = (tensor(4008, t, (B, N, Hq, d), torch.bfloat16) for t in (1, 4))
    k, v = (tensor(4008, t, (B, N, H, d), torch.bfloat16) for t in (2, 3))
    freqs = fa.rope_frequencies(rot, 10000.0, "linear", 4.0)
    pos = torch.arange(5000, 5000 + N, dtype=torch.int32, device="cuda").view(B, N)
    tq, tk = fa.rope(q, k, freqs, pos, interleaved=True)
    o, lse = fa.forward(tq, tk, v, causal=True)
    gq, gk, gv = fa.backward(tq, tk, v, o, lse, dy, causal=True)
    gq, gk = fa.rope_backward(gq, gk, freqs, pos, interleaved=True)
    w, p = freqs.cpu().numpy(), pos.cpu().numpy().reshape(-1)
    turn = lambda x, h, back: turn64(x.reshape(N, h, d), p, w, rot, True, 1.0, back)[0].reshape(B, N, h, d)  # noqa: E731
    rq, rk, rv = orc.attention_bwd(turn(host64(q), Hq, False), turn(host64(k), H, False), host64(v), host64(dy),
                                   d ** -0.5, causal=True)
    check_grad(host64(gq), turn(np.asarray(rq, np.float64), Hq, True), "dQ")
    check_grad(host64(gk), turn(np.asarray(rk, np.float64), H, True), "dK")
    check_grad(host64(gv), np.asarray(rv, np.float64), "dV")


def test_rope_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are those of a small call."""
    N = (1 << 31) // (64 * 128) + 100
    q = torch.zeros(N, 64, 128, dtype=torch.bfloat16, device="cuda")
    tail = tensor(4009, si.Q, (100, 64, 128), torch.bfloat16)
    q[-100:] = tail
    freqs = fa.rope_frequencies(128)
    want, _ = fa.rope(tail, None, freqs, torch.arange(N - 100, N, dtype=torch.int32, device="cuda"))
    fa.rope(q, None, freqs, q_out=q)
    assert torch.equal(q[-100:], want) and not q[:-100:9973].any()


def test_rope_on_another_stream_and_captured():
    q, k = tensor(4007, si.Q, (40, 8, 128), torch.bfloat16), tensor(4007, si.K, (40, 2, 128), torch.bfloat16)
    freqs = fa.rope_frequencies(128)
    want = fa.rope(q, k, freqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = fa.rope(q, k, freqs)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.rope(q, k, freqs, q_out=yq, k_out=yk)
    q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    # doubling is exact, so the captured call on the new values gives exactly twice the old
    assert torch.equal(yq, want[0] * 2) and torch.equal(yk, want[1])


def test_rope_empty_batch():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = fa.rope(q, None, fa.rope_frequencies(64))
    assert y.shape == q.shape

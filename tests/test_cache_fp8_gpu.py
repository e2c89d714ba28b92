"""The e4m3 paged cache on the GPU: fa_cache_append_fp8 bit for bit against the 64-bit model of
cache8.py (scales are powers of two, so nothing else is rounded than the codes, to nearest even),
and fa_decode_paged_fp8 against attention in 64 bits over the stored values.

Tolerance of o: half a bf16 step of the value (2^-8); of the weights p * scale 2^-11 relative (fp16)
or 2^-25 of the largest one below fp16's normal range, so 2^-11 sum p|v| + 2^-25 sum|v|; and 2^-17
(1 + t) relative for the fp32 scores (d = 128 products of size t in all, 2^-24 each, and the fp32
exponentials).  lse: 2^-17 (1 + t).

More than 16 query rows of a K/V head at d = 128 take the kernel that multiplies e4m3 bytes, with q and
the weights as two e4m3 terms.  Weights: the first term is off by at most 2^-4 of the weight and the
second by 2^-4 of that, 2^-8 together, where its 16-fold is normal; below, by half of 2^-9 / 16 = 2^-14
while the largest weight of the row is at least 2^2, so by 2^-16 of it: 2^-16 sum|v| times the
largest over the smallest scale.  q: exact down to the step of the second term, 2^-9 where the
row's largest element is at least 2^7, so off by at most 2^-17 of that element: 2^-17 u for scores,
with u = max|q| sum|k| scale in place of t = sum|q||k| scale."""
import math

import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


def check(o, lse, ref, q, kv):
    """kv: the cache's (codes, scales) of K and V and table, lens, sb, scale of cache8.attend."""
    r_o, r_lse, o_abs, v_sum, t_abs = ref
    got = o.double().cpu().numpy().reshape(r_o.shape)
    gl = lse.double().cpu().numpy().reshape(r_lse.shape)
    assert not np.isnan(got).any()
    weight, small, u = 2.0 ** -11, 2.0 ** -25, 0.0
    q64 = q.double().cpu().numpy().reshape(r_o.shape)
    _, Nq, Hq, d = q64.shape
    if Nq * Hq // kv[0].shape[2] > 16 and d == 128:
        used = kv[3][np.isfinite(kv[3]) & (kv[3] > 0)]
        weight, small = 2.0 ** -8, 2.0 ** -16 * used.max() / used.min()
        u = _score_bound(q64, kv)
    t = t_abs + u
    tt = t.transpose(0, 2, 1)[..., None]
    tol = 2.0 ** -8 * np.abs(r_o) + (weight + 2.0 ** -17 * (1 + tt)) * o_abs + small * v_sum
    bad = np.abs(got - r_o) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], np.abs(got - r_o).max())
    none = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(gl), none)
    assert np.all(np.abs(gl[~none] - r_lse[~none]) <= 2.0 ** -17 * (1 + t[~none]))


def _score_bound(q, kv):
    """max|q| times the largest sum|k| of the sequence, times the scale: [B, Hq, Nq]."""
    kc, ks, _, _, table, lens, sb, scale = kv
    B, Nq, Hq, _ = q.shape
    out = np.zeros((B, Hq, Nq))
    for b in range(B):
        if lens[b] == 0:
            continue
        k = np.abs(cache8.gather(kc, ks, table[b], lens[b], sb)).sum(-1).max(0)  # [H]
        out[b] = np.abs(q[b]).max(-1).T * np.repeat(k, Hq // kc.shape[2])[:, None] * scale
    return out


CASES = [
    # lens, Nq, Hq, Hkv, d, page_size, scale_block
    ([1], 1, 1, 1, 64, 16, 16),
    ([37, 0, 16], 1, 12, 12, 64, 16, 16),
    ([1000, 1, 0, 333, 64], 1, 32, 4, 128, 16, 16),
    ([65, 64, 700], 1, 16, 2, 64, 32, 16),
    ([2047, 130], 1, 8, 8, 128, 64, 32),
    ([1, 127, 128, 129, 900], 1, 64, 4, 128, 128, 128),
    ([700, 300], 1, 40, 2, 128, 256, 64),       # 20 heads of a group
    ([513, 512], 1, 33, 1, 64, 512, 256),       # 33 heads of a group
    ([300, 5, 0, 2, 129], 5, 16, 2, 128, 16, 16),  # new tokens that see nothing
    ([64, 65, 66], 3, 7, 1, 64, 32, 32),
    ([400, 70], 9, 12, 4, 128, 64, 64),
    ([150, 40], 40, 4, 2, 64, 64, 16),
    ([3000, 10], 2, 8, 1, 128, 16, 16),
    ([200, 70], 20, 8, 2, 128, 32, 16),         # 80 query rows of a head: two tiles, the second part full
    ([33, 1000], 1, 17, 1, 128, 16, 16),
    ([129, 257], 16, 8, 2, 128, 64, 64),        # 64 rows: a full tile
    ([100] * 90, 3, 12, 2, 128, 16, 16),        # more short units than CTAs
    ([40, 0, 3] * 40, 1, 8, 4, 128, 16, 16),
    ([520] * 30, 1, 6, 6, 64, 16, 16),
    ([300, 40, 0, 2], 3, 16, 4, 64, 32, 16),    # 9 to 16 rows: four, two and one K/V heads at a time
    ([700, 33], 2, 14, 2, 64, 16, 16),
    ([513, 12], 11, 2, 2, 128, 64, 64),
    ([260, 259], 1, 12, 1, 64, 64, 32),
    ([290, 7, 5], 8, 3, 3, 128, 32, 32),        # 8 new tokens, each its own row
    ([1030, 4], 4, 4, 2, 128, 512, 256),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{'_'.join(map(str, c[0]))}-n{c[1]}-h{c[2]}_{c[3]}-d{c[4]}-p{c[5]}_{c[6]}"
                                             for c in CASES])
def test_decode_fp8_matches_64_bits(case):
    lens, Nq, Hq, H, d, ps, sb = case
    rng = np.random.default_rng(5001)
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), Nq, Hq, d))).cuda().bfloat16()
    dkc, dks, dvc, dvs, dt, dl = cache8.to_device(kc, ks, vc, vs, table, lens)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d))
    ws = torch.full((fa.fa_decode_paged_fp8_workspace_size(len(lens), Nq, Hq, H, d),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    o, lse = fa.decode_paged_fp8(q, dkc, dvc, dks, dvs, dt, dl, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == fa.FA_OK
    check(o, lse, ref, q, (kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d)))
    # the workspace, used once, gives the same bits again; so does the 3-D form for one token
    o2, lse2 = fa.decode_paged_fp8(q if Nq > 1 else q[:, 0], dkc, dvc, dks, dvs, dt, dl, workspace=ws)
    assert torch.equal(o2.view_as(o), o) and torch.equal(lse2.view_as(lse), lse)


@pytest.mark.parametrize("Hq", [8, 48], ids=["4rows", "24rows"])
@pytest.mark.parametrize("sb", [16, 64])
def test_decode_fp8_scales_of_very_different_size(sb, Hq):
    """V scales from 2^-40 to 2^30 and K scales that swamp some blocks: weights are taken relative
    to the largest product of probability and scale, so the small blocks keep their bits."""
    rng = np.random.default_rng(5002)
    lens, H, d, ps = [400, 77], 2, 128, 64
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, spread=0.0)
    vs *= np.exp2(rng.integers(-40, 31, vs.shape))
    ks *= np.exp2(rng.integers(-6, 2, ks.shape))
    # the block with the largest scale is one that softmax gives nothing
    for b in range(2):
        vs[table[b, 0], :, 0] = 2.0 ** 30
        ks[table[b, 0], :, 0] = 0.0
    q = torch.from_numpy(rng.standard_normal((2, 1, Hq, d)) * 4).cuda().bfloat16()
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1.0)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=1.0)
    r_o, r_lse, o_abs, v_sum, t_abs = ref
    got = o.double().cpu().numpy()
    n = np.array(lens).reshape(2, 1, 1, 1)
    # a small weight is off by 2^-25 of the largest one (fp16) or 2^-16 (two e4m3 terms), times a code
    # of at most 448
    weight, small = (2.0 ** -11, 2.0 ** -25) if Hq // H <= 16 else (2.0 ** -8, 2.0 ** -16)
    q64 = q.double().cpu().numpy()
    u = 0.0 if Hq // H <= 16 else _score_bound(q64, (kc, ks, vc, vs, table, lens, sb, 1.0))
    wsum = _weight_max(q64, kc, ks, vs, table, lens, sb)
    tt = (t_abs + u).transpose(0, 2, 1)[..., None]
    tol = 2.0 ** -8 * np.abs(r_o) + (weight + 2.0 ** -17 * (1 + tt)) * o_abs + n * small * 448 * wsum
    assert np.all(np.abs(got - r_o) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - r_lse) <= 2.0 ** -17 * (1 + t_abs + u))


@pytest.mark.parametrize("Hq", [4, 40], ids=["4rows", "40rows"])
@pytest.mark.parametrize("way", ["up", "down", "steps"])
def test_decode_fp8_scores_that_rise_and_fall(way, Hq):
    """K scales that double every few blocks: running maxima move in most chunks, or never again."""
    rng = np.random.default_rng(5016)
    lens, H, d, ps, sb = [1500, 700], 1, 128, 32, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, spread=0.5)
    for b, n in enumerate(lens):
        j = np.arange(n // sb + (n % sb > 0)) * sb
        at = np.linspace(0, 1, len(j))
        grow = {"up": 9 * at, "down": 9 * at[::-1], "steps": np.round(6 * np.sin(20 * at))}[way]
        ks[table[b, j // ps], :, j % ps // sb] *= np.exp2(np.round(grow))[:, None]
    q = torch.from_numpy(rng.standard_normal((2, 1, Hq, d))).cuda().bfloat16()
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d))
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
    check(o, lse, ref, q, (kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d)))


@pytest.mark.parametrize("Hq", [4, 40], ids=["4rows", "40rows"])
@pytest.mark.parametrize("e", [-100, 100])
def test_decode_fp8_scales_that_queries_undo(e, Hq):
    """K scales times 2^e and queries times 2^-e change no bit (powers of two round nothing); V scales
    times 2^(e / 2) scale o, the references t + log2(scale) being rounded at 64 at most (2^-18)."""
    rng = np.random.default_rng(5017)
    lens, H, d, ps, sb = [300, 41], 1, 128, 32, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((2, 1, Hq, d))).cuda().bfloat16()
    dkc, dks, dvc, dvs, dt, dl = cache8.to_device(kc, ks, vc, vs, table, lens)
    o, lse = fa.decode_paged_fp8(q, dkc, dvc, dks, dvs, dt, dl)
    q2 = (q.float() * 2.0 ** -e).bfloat16()
    o2, lse2 = fa.decode_paged_fp8(q2, dkc, dvc, dks * 2.0 ** e, dvs, dt, dl)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    vs = vs * 2.0 ** (e // 2)
    o2, lse2 = fa.decode_paged_fp8(q, dkc, dvc, dks, dvs * 2.0 ** (e // 2), dt, dl)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d))
    check(o2, lse2, ref, q, (kc, ks, vc, vs, table, lens, sb, 1 / math.sqrt(d)))


def _weight_max(q, kc, ks, vs, table, lens, sb):
    """Largest p_j * scale_j / sum p of each query, [B, 1, Hq, 1]."""
    B, _, Hq, _ = q.shape
    H, ps = kc.shape[2], kc.shape[1]
    out = np.zeros((B, 1, Hq, 1))
    for b in range(B):
        k = cache8.gather(kc, ks, table[b], lens[b], sb)
        j = np.arange(lens[b])
        s = vs[table[b, j // ps], :, j % ps // sb]
        for h in range(Hq):
            t = k[:, h // (Hq // H)] @ q[b, 0, h]
            p = np.exp(t - t.max())
            out[b, 0, h] = (p * s[:, h // (Hq // H)]).max() / p.sum()
    return out


def test_decode_fp8_extreme_queries_and_zero_scales():
    """Queries of 2^-60 and 2^60 times a scale that undoes it, a zero query (mean of V), K scale 0."""
    rng = np.random.default_rng(5003)
    lens, H, d, ps, sb = [90], 1, 64, 16, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, spread=0.5)
    ks[table[0, 1], 0, 0] = 0.0
    base = rng.standard_normal((1, 1, 3, d))
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    for e in (-60, 0, 60):
        q = torch.from_numpy(base).cuda().bfloat16()
        q[:, :, 2] = 0
        q = (q.float() * 2.0 ** e).bfloat16()
        scale = 0.125 * 2.0 ** -e
        ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, scale)
        o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=scale)
        check(o, lse, ref, q, (kc, ks, vc, vs, table, lens, sb, scale))


def test_decode_fp8_nan_reaches_only_what_attends_to_it():
    rng = np.random.default_rng(5004)
    lens, H, d, ps, sb = [40, 40], 2, 64, 16, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d)
    q = torch.from_numpy(rng.standard_normal((2, 4, d))).cuda().bfloat16()
    clean = cache8.to_device(kc, ks, vc, vs, table, lens)
    o0, l0 = fa.decode_paged_fp8(q, clean[0], clean[2], clean[1], clean[3], clean[4], clean[5])
    for w in ("k code", "v code", "k scale", "v scale"):
        a = [kc.copy(), ks.copy(), vc.copy(), vs.copy()]
        page = table[0, 1]
        if w == "k code":
            a[0][page, 3, 1, 5] = 0x7F
        elif w == "v code":
            a[2][page, 3, 1, 5] = 0xFF
        elif w == "k scale":
            a[1][page, 1, 0] = np.nan
        else:
            a[3][page, 1, 0] = np.nan
        dev = cache8.to_device(*a, table, lens)
        o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
        # heads 2, 3 of sequence 0 read K/V head 1; a V code spoils its column only
        assert torch.isnan(o[0, 2:]).all() if w != "v code" else torch.isnan(o[0, 2:, 5]).all(), w
        assert torch.equal(o[0, :2], o0[0, :2]) and torch.equal(o[1], o0[1]), w
        if w.startswith("k"):
            assert torch.isnan(lse[0, 2:]).all(), w
        else:
            assert torch.equal(lse, l0), w
    assert fa.fa_last_device_error() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 8, 24], ids=["8rows", "16rows", "48rows"])
def test_decode_fp8_nan_of_a_later_token_is_not_seen_before_it(Hq, d):
    """Four new tokens; the third one's V row holds a NaN code, the last one's block scale is NaN."""
    rng = np.random.default_rng(5011)
    lens, H, ps, sb, Nq = [49], 2, 16, 16, 4
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d)
    q = torch.from_numpy(rng.standard_normal((1, Nq, Hq, d))).cuda().bfloat16()
    clean = cache8.to_device(kc, ks, vc, vs, table, lens)
    o0, l0 = fa.decode_paged_fp8(q, clean[0], clean[2], clean[1], clean[3], clean[4], clean[5])
    vc[table[0, 2], 15, 0, 57] = 0x7F  # token 47, K/V head 0, one column
    vs[table[0, 3], 1, 0] = np.nan     # token 48, K/V head 1
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
    want = torch.zeros(1, Nq, Hq, d, dtype=torch.bool, device="cuda")
    want[0, 2:, :Hq // 2, 57] = True
    want[0, 3, Hq // 2:] = True
    assert torch.equal(torch.isnan(o), want)
    assert torch.equal(o[~want], o0[~want]) and torch.equal(lse, l0)


def test_decode_fp8_reports_bad_page_and_clamps_lengths():
    rng = np.random.default_rng(5005)
    lens, H, d, ps, sb = [60, 30], 1, 64, 16, 16
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d)
    q = torch.from_numpy(rng.standard_normal((2, 4, d))).cuda().bfloat16()
    dev = cache8.to_device(kc, ks, vc, vs, table, [60, -7])
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
    assert torch.all(o[1] == 0) and torch.isneginf(lse[1]).all() and fa.fa_last_device_error() == fa.FA_OK
    bad = table.copy()
    bad[1, 1] = kc.shape[0]
    dev = cache8.to_device(np.zeros_like(kc), np.zeros_like(ks), np.zeros_like(vc), np.zeros_like(vs), bad, lens)
    fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
    assert fa.fa_last_device_error() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_last_device_error() == fa.FA_OK


APPENDS = [
    # old lengths, new lengths, Hkv, d, page_size, scale_block
    ([0], [1], 1, 64, 16, 16),
    ([15, 16, 17, 0], [1, 1, 1, 1], 8, 128, 16, 16),
    ([0, 5, 31, 40], [100, 0, 33, 7], 3, 128, 32, 16),
    ([3, 0], [300, 129], 2, 64, 64, 64),
    ([200, 0, 1], [60, 256, 700], 5, 128, 256, 256),
    ([127, 128], [2, 1], 4, 64, 128, 128),
    ([9] * 40, [3] * 40, 1, 128, 16, 16),
]


def _append_problem(rng, old, new, H, d, ps, sb, grow=1.0):
    lens = [a + b for a, b in zip(old, new)]
    kc, ks, vc, vs, table = cache8.build(rng, old, ps, sb, H, d, extra=0)
    need = sum((n + ps - 1) // ps for n in lens) + 2
    P = kc.shape[0]
    extra = need - P + 1

    def pad(a, v):
        return np.concatenate([a, np.full((max(extra, 0), *a.shape[1:]), v, a.dtype)])
    kc, vc, ks, vs = pad(kc, 0x7F), pad(vc, 0x7F), pad(ks, np.nan), pad(vs, np.nan)
    free = [p for p in range(kc.shape[0]) if p not in set(table[table >= 0].tolist())]
    full = np.full((len(lens), max((n + ps - 1) // ps for n in lens) + 1), -1, np.int32)
    for b, n in enumerate(lens):
        had = (old[b] + ps - 1) // ps
        full[b, :had] = table[b, :had]
        for t in range(had, (n + ps - 1) // ps):
            full[b, t] = free.pop()
    total = sum(new)
    xs = []
    for _ in range(2):
        x = rng.standard_normal((total, H, d)) * np.exp2(rng.uniform(-3, 3, (total, H, 1))) * grow
        xs.append(torch.from_numpy(x).bfloat16())
    return kc, ks, vc, vs, full, lens, xs


def _run_append(kc, ks, vc, vs, table, lens, cu, xs):
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    fa.cache_append_fp8(xs[0].cuda(), xs[1].cuda(), dev[0], dev[2], dev[1], dev[3], dev[4], dev[5],
                        None if cu is None else torch.from_numpy(np.array(cu, np.int32)).cuda())
    torch.cuda.synchronize()
    return dev


def _same(dev, kc, ks, vc, vs):
    for t, a in ((dev[0], kc), (dev[2], vc)):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), a)
    for t, a in ((dev[1], ks), (dev[3], vs)):
        np.testing.assert_array_equal(t.cpu().numpy().astype(np.float64), a.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("grow", [0.01, 1.0, 1e4], ids=["smaller", "alike", "larger"])
@pytest.mark.parametrize("case", APPENDS, ids=[f"{len(c[0])}seq_{sum(c[1])}new_p{c[4]}_{c[5]}" for c in APPENDS])
def test_append_is_the_model_bit_for_bit(case, grow):
    old, new, H, d, ps, sb = case
    kc, ks, vc, vs, table, lens, xs = _append_problem(np.random.default_rng(5006), old, new, H, d, ps, sb, grow)
    cu = [0] + np.cumsum(new).tolist()
    dev = _run_append(kc, ks, vc, vs, table, lens, cu, xs)
    for codes, scales, x in ((kc, ks, xs[0]), (vc, vs, xs[1])):
        cache8.append(codes, scales, x.double().numpy(), table, lens, cu, sb)
    _same(dev, kc, ks, vc, vs)
    assert fa.fa_last_device_error() == fa.FA_OK
    if all(n == 1 for n in new):  # without offsets: one row each, the same bits
        kc2, ks2, vc2, vs2, table2, lens2, xs2 = _append_problem(np.random.default_rng(5006), old, new, H, d, ps, sb,
                                                                 grow)
        _same(_run_append(kc2, ks2, vc2, vs2, table2, lens2, None, xs2), kc, ks, vc, vs)


def test_append_rows_before_and_after_the_sequences():
    """Offsets may start past 0 and end before the last row: those rows belong to no sequence."""
    rng = np.random.default_rng(5012)
    old, new, H, d, ps, sb = [3, 0, 40], [2, 35, 1], 2, 128, 32, 16
    kc, ks, vc, vs, table, lens, xs = _append_problem(rng, old, new, H, d, ps, sb)
    junk = [torch.full((n, H, d), float("nan"), dtype=torch.bfloat16) for n in (77, 50)]
    cu = [77, 79, 114, 115]
    dev = _run_append(kc, ks, vc, vs, table, lens, cu, [torch.cat([junk[0], x, junk[1]]) for x in xs])
    for codes, scales, x in ((kc, ks, xs[0]), (vc, vs, xs[1])):
        cache8.append(codes, scales, x.double().numpy(), table, lens, [0, 2, 37, 38], sb)
    _same(dev, kc, ks, vc, vs)
    assert fa.fa_last_device_error() == fa.FA_OK


def test_append_special_values():
    """Zeros, signed zeros, the type's extremes, subnormals, and rows that are not finite."""
    rng = np.random.default_rng(5007)
    old, new, H, d, ps, sb = [5, 0, 3], [20, 16, 2], 2, 64, 32, 16
    kc, ks, vc, vs, table, lens, xs = _append_problem(rng, old, new, H, d, ps, sb)
    big = float(torch.finfo(torch.bfloat16).max)
    xs[0][:3] = 0.0
    xs[0][1, 0] = -0.0
    xs[0][3, 1, 7] = big
    xs[0][12, 0, 0] = -big
    xs[1][:20] = torch.tensor(2.0 ** -133).bfloat16() * torch.sign(xs[1][:20].float()).bfloat16()
    xs[1][20:36, 0] = 0.0
    xs[1][36, 0, 1] = float("nan")
    xs[1][37, 1, 2] = float("inf")
    cu = [0, 20, 36, 38]
    dev = _run_append(kc, ks, vc, vs, table, lens, cu, xs)
    for codes, scales, x in ((kc, ks, xs[0]), (vc, vs, xs[1])):
        cache8.append(codes, scales, x.double().numpy(), table, lens, cu, sb)
    _same(dev, kc, ks, vc, vs)
    assert np.isnan(vs[table[2, 0], :, 0]).all()


def test_append_token_by_token_reads_like_at_once():
    """Power-of-two scales: a code that was rescaled differs from one written at once only below
    the smallest normal e4m3 value (2^-6 of its scale), by at most half a step there each time the
    scale grew (2^-10 of the final scale each, under 2^-9 in all)."""
    rng = np.random.default_rng(5008)
    H, d, ps, sb, n = 2, 128, 32, 32, 70
    kc, ks, vc, vs, table, lens, xs = _append_problem(rng, [0], [n], H, d, ps, sb)
    once = _run_append(kc, ks, vc, vs, table, lens, [0, n], xs)
    step = cache8.to_device(kc, ks, vc, vs, table, lens)
    k, v = xs[0].cuda(), xs[1].cuda()
    for i in range(n):
        at = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        fa.cache_append_fp8(k[i:i + 1], v[i:i + 1], step[0], step[2], step[1], step[3], step[4], at)
    assert torch.equal(once[1].nan_to_num(-1), step[1].nan_to_num(-1))
    for w in (0, 2):
        a, b = (cache8.gather(x[w].view(torch.uint8).cpu().numpy(), x[w + 1].double().cpu().numpy(), table[0], n, sb)
                for x in (once, step))
        s = np.repeat(once[w + 1].double().cpu().numpy()[table[0, :3], :, 0], 32, 0)[:n][..., None]
        assert np.all(np.abs(a - b) <= 2.0 ** -9 * s)
        assert np.all((a == b) | (np.abs(a) < 2.0 ** -5 * s))


def test_append_skips_and_records_what_it_cannot_use():
    rng = np.random.default_rng(5009)
    H, d, ps, sb = 1, 64, 16, 16
    for what in ("length", "page", "offsets", "table"):
        kc, ks, vc, vs, table, lens, xs = _append_problem(rng, [4, 20], [3, 30], H, d, ps, sb)
        cu, mlens, mtable = [0, 3, 33], list(lens), table.copy()
        if what == "length":
            mlens[0] = 2  # fewer than the 3 new rows
        elif what == "page":
            mtable[0, 0] = kc.shape[0] + 5
        elif what == "table":
            mlens[0] = table.shape[1] * ps + 1
        else:
            cu = [5, 3, 33]
        dev = _run_append(kc, ks, vc, vs, mtable, mlens, cu, xs)
        assert fa.fa_last_device_error() == fa.FA_ERR_INVALID_ARG, what
        for codes, scales, x in ((kc, ks, xs[0]), (vc, vs, xs[1])):  # the second sequence is served
            cache8.append(codes, scales, x.double().numpy(), table, [0, lens[1]], [3, 3, 33], sb)
        _same(dev, kc, ks, vc, vs)
    assert fa.fa_last_device_error() == fa.FA_OK


@pytest.mark.parametrize("Nq", [1, 3], ids=["16rows", "24rows"])
def test_cache_past_32_bit_offsets(Nq):
    """A pool of more than 2^32 bytes: a sequence in its last pages gives the bits that it gives in a
    small pool, appended and read."""
    rng = np.random.default_rng(5013)
    lens, H, d, ps, sb = [150], 8, 128, 64, 16
    kc, ks, vc, vs, table, lens, xs = _append_problem(rng, [100], [50], H, d, ps, sb)
    cu = [0, 50]
    q = torch.from_numpy(rng.standard_normal((1, Nq, 64, d))).cuda().bfloat16()
    small = _run_append(kc, ks, vc, vs, table, lens, cu, xs)
    want = fa.decode_paged_fp8(q, small[0], small[2], small[1], small[3], small[4], small[5])
    P = (1 << 32) // (ps * H * d) + 10
    base = P - kc.shape[0]
    big = []
    for host in (kc, ks, vc, vs):
        t = torch.zeros(P, *host.shape[1:], dtype=torch.uint8 if host.dtype == np.uint8 else torch.float32, device="cuda")
        t[base:] = torch.from_numpy(host.astype(np.uint8 if host.dtype == np.uint8 else np.float32)).cuda()
        big.append(t)
    t = torch.from_numpy(np.where(table >= 0, table + base, -1).astype(np.int32)).cuda()
    fa.cache_append_fp8(xs[0].cuda(), xs[1].cuda(), big[0], big[2], big[1], big[3], t, small[5],
                        torch.tensor(cu, dtype=torch.int32, device="cuda"))
    got = fa.decode_paged_fp8(q, big[0], big[2], big[1], big[3], t, small[5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(big[0][base:], small[0].view(torch.uint8)) and not big[0][:base:997].any()
    # and its pages move: compaction brings them to the front
    t2, n = fa.pages_compact([*big], t, small[5], ps)
    assert int(n) == 3 and int(t2.max()) <= 2
    got = fa.decode_paged_fp8(q, big[0], big[2], big[1], big[3], t2, small[5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.fa_last_device_error() == fa.FA_OK


def test_decode_fp8_two_streams_at_once():
    """Calls with workspaces of their own do not disturb one another, nor does a captured one."""
    rng = np.random.default_rng(5014)
    jobs = []
    for lens, Nq, Hq, H, d in (([700, 20, 300], 1, 16, 4, 128), ([900, 64], 4, 8, 1, 128), ([500], 2, 4, 2, 64)):
        kc, ks, vc, vs, table = cache8.build(rng, lens, 32, 16, H, d)
        dev = cache8.to_device(kc, ks, vc, vs, table, lens)
        q = torch.from_numpy(rng.standard_normal((len(lens), Nq, Hq, d))).cuda().bfloat16()
        jobs.append((q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5]))
    want = [fa.decode_paged_fp8(*j) for j in jobs]
    graphs = []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fa.decode_paged_fp8(*j)
        graphs.append((g, out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    got = []
    for i in range(30):
        with torch.cuda.stream(streams[i % 3]):
            got.append((i % 3, fa.decode_paged_fp8(*jobs[i % 3])))
        if i % 5 == 0:
            with torch.cuda.stream(streams[3 + i % 3]):
                graphs[i % 3][0].replay()
    torch.cuda.synchronize()
    got += [(i, out) for i, (_, out) in enumerate(graphs)]
    for i, (o, lse) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_c_functions_by_their_names():
    """The C functions through the binding's functions of the same names give what the helpers give."""
    rng = np.random.default_rng(5015)
    old, new, H, d, ps, sb = [20, 0], [13, 40], 2, 64, 32, 16
    kc, ks, vc, vs, table, lens, xs = _append_problem(rng, old, new, H, d, ps, sb)
    cu, P, maxp = [0, 13, 53], kc.shape[0], table.shape[1]
    want = _run_append(kc, ks, vc, vs, table, lens, cu, xs)
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    fa.fa_cache_append_fp8(xs[0].cuda(), xs[1].cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"), dev[4], dev[5],
                           dev[0], dev[2], dev[1], dev[3], 2, 53, H, P, ps, maxp, sb, d)
    for a, b in zip(dev, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q = torch.from_numpy(rng.standard_normal((2, 3, 4, d))).cuda().bfloat16()
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=0.25)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    n = fa.fa_decode_paged_fp8_workspace_size(2, 3, 4, H, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    fa.fa_decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], o2, lse2, 2, 3, 4, H, P, ps, maxp, sb, d,
                           0.25, ws, n)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    freqs = fa.rope_frequencies(32)
    y, _ = fa.rope(q, None, freqs)
    y2 = torch.empty_like(y)
    fa.fa_rope(q, None, y2, None, None, freqs, 6, 3, 4, 0, d, 32, False, 1.0, False, fa.FA_BF16, 4 * d, 0, 4 * d, 0)
    assert torch.equal(y, y2)
    parent = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
    pools = [dev[0], dev[1], dev[2], dev[3]]
    room = [torch.cat([t, t[:2]]) for t in pools]  # two free pages more
    got = fa.pages_fork(room, dev[4], dev[5], parent, ps)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    t2, l2, f2, c2 = i32(3, maxp), i32(3), i32(P + 2), i32(1)
    n = fa.fa_pages_workspace_size(P + 2, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    raw = [(t.data_ptr(), t.nbytes // (P + 2)) for t in room]
    fa.fa_pages_fork(raw, dev[4], dev[5], parent, t2, l2, f2, c2, 2, 3, P + 2, ps, maxp, ws, n)
    for a, b in zip(got, (t2, l2, f2, c2)):
        assert torch.equal(a, b)
    t3, n3 = fa.pages_compact(room, t2, l2, ps)
    t4, n4 = i32(3, maxp), i32(1)
    fa.fa_pages_compact(room, t2, l2, t4, n4, 3, P + 2, ps, maxp, ws, n)
    assert torch.equal(t3, t4) and torch.equal(n3, n4)
    assert fa.fa_last_device_error() == fa.FA_OK


def test_prefill_then_decode_through_the_cache():
    """The whole path: rope, forward, append of the prompt, then steps of rope, append and decode,
    against attention in 64 bits over what the cache holds; once more through a captured graph on
    another stream."""
    rng = np.random.default_rng(5010)
    H, Hq, d, ps, sb, steps = 2, 8, 128, 32, 16, 5
    new = [50, 1, 64]
    lens = list(new)
    maxp = 4
    table = rng.permutation(3 * maxp).reshape(3, maxp).astype(np.int32)
    P = 3 * maxp
    kp = torch.full((P, ps, H, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vp = kp.clone()
    ks = torch.full((P, H, ps // sb), float("nan"), device="cuda")
    vs = ks.clone()
    dt = torch.from_numpy(table).cuda()
    freqs = fa.rope_frequencies(d, 10000.0, "linear", 2.0)
    cu = torch.tensor([0, 50, 51, 115], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in new]).int().cuda()
    q, k, v = (torch.from_numpy(rng.standard_normal((115, h, d))).cuda().bfloat16() for h in (Hq, H, H))
    q, k = fa.rope(q, k, freqs, pos)
    fa.forward(q, k, v, causal=True, cu_seqlens=cu)
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fa.cache_append_fp8(k, v, kp, vp, ks, vs, dt, seqlens, cu)

    sq, sk, sv = (torch.zeros(3, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))

    def step():
        seqlens.add_(1)
        a, b = fa.rope(sq, sk, freqs, seqlens - 1)
        fa.cache_append_fp8(b, sv, kp, vp, ks, vs, dt, seqlens)
        return (a, *fa.decode_paged_fp8(a, kp, vp, ks, vs, dt, seqlens))

    def verify(a, o, lse):
        ln = seqlens.cpu().numpy()
        cache = (kp.view(torch.uint8).cpu().numpy(), ks.double().cpu().numpy(), vp.view(torch.uint8).cpu().numpy(),
                 vs.double().cpu().numpy(), table, ln, sb, 1 / math.sqrt(d))
        ref = cache8.attend(a.double().cpu().numpy()[:, None], *cache)
        check(o[:, None], lse[..., None], ref, a, cache)

    def feed():
        for t in (sq, sk, sv):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape))))

    for _ in range(steps):
        feed()
        verify(*step())
    g = torch.cuda.CUDAGraph()
    was = seqlens.clone()
    with torch.cuda.graph(g):
        out = step()
    seqlens.copy_(was)
    for _ in range(3):
        feed()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        verify(*out)
    assert fa.fa_last_device_error() == fa.FA_OK


def test_captured_after_copies_and_joined_streams():
    """Launches may come early, while what is before them in the stream ends: in a captured graph
    that can be a copy, a fill, or the join of two streams.  Every replay reads what came before it."""
    B, H, Hq, d, ps, sb, maxp = 3, 2, 48, 128, 32, 16, 2
    P = B * maxp + 4
    src = [torch.randn(B, h, d, device="cuda").bfloat16() for h in (Hq, H, H)]
    q, k, v = (torch.zeros_like(t) for t in src)
    kp, vp = (torch.zeros(P, ps, H, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(P, H, ps // sb, device="cuda") for _ in range(2))
    dt = torch.arange(B * maxp, dtype=torch.int32, device="cuda").view(B, maxp)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    parent = torch.tensor([2, 2, 0], dtype=torch.int32, device="cuda")
    freqs = fa.rope_frequencies(d)
    side = torch.cuda.Stream()

    def chain():
        q.copy_(src[0])  # a copy straight before the rotation
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            k.copy_(src[1])
            v.copy_(src[2])
            fa.rope(k, None, freqs, lens, q_out=k)
        fa.rope(q, None, freqs, lens, q_out=q)
        torch.cuda.current_stream().wait_stream(side)  # both streams before the append
        lens.add_(1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lens2 = lens.clone()
        torch.cuda.current_stream().wait_stream(side)
        fa.cache_append_fp8(k, v, kp, vp, ks, vs, dt, lens2)
        o, lse = fa.decode_paged_fp8(q, kp, vp, ks, vs, dt, lens)
        table, ln, free, n = fa.pages_fork([kp, vp, ks, vs], dt, lens, parent, ps)
        o2, lse2 = fa.decode_paged_fp8(q, kp, vp, ks, vs, table, ln)
        return o, lse, table, ln, free, n, o2, lse2

    def fresh(n):
        for t in src:
            t.copy_(torch.randn(t.shape, device="cuda"))
        for t in (kp.view(torch.uint8), vp.view(torch.uint8), ks, vs, lens):
            t.zero_()
        lens.fill_(n)

    state = torch.cuda.get_rng_state()
    want = []
    for n in (0, 17, 30):
        fresh(n)
        want.append([t.clone() for t in chain()])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain()
    torch.cuda.set_rng_state(state)
    for n, w in zip((0, 17, 30), want):
        fresh(n)
        g.replay()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
    assert torch.isfinite(out[0].float()).all() and fa.fa_last_device_error() == fa.FA_OK


@pytest.mark.parametrize("Hq,Nq", [(8, 1), (32, 1), (64, 3)], ids=["1row", "4rows", "24rows"])
def test_calls_back_to_back_repeat_bit_for_bit(Hq, Nq):
    """A chain in which every call reads what the one before wrote, many times without a pause: a call
    that began before its inputs were complete would differ."""
    B, H, d, ps, sb, maxp = 6, 8, 128, 16, 16, 40
    P = B * maxp + 8
    lens0 = torch.tensor([600, 1, 333, 17, 500, 64], dtype=torch.int32, device="cuda")
    total = int(lens0.sum())
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens0.cumsum(0).int()])
    pos = torch.cat([torch.arange(n) for n in lens0.tolist()]).int().cuda()
    k0, v0 = (torch.randn(total, H, d, device="cuda").bfloat16() for _ in range(2))
    q0 = torch.randn(B * Nq, Hq, d, device="cuda").bfloat16()
    qpos = (lens0[:, None] - Nq + torch.arange(Nq, device="cuda").int()).reshape(-1).int().contiguous()
    freqs = fa.rope_frequencies(d)
    table = torch.randperm(P, device="cuda")[:B * maxp].int().view(B, maxp)
    parent = torch.tensor([5, 0, 0, 2, 4, 0], dtype=torch.int32, device="cuda")
    pages = [torch.zeros(P, ps, H, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(P, H, ps // sb, device="cuda") for _ in range(2)]
    first = None
    for turn in range(60):
        for t in (*pages, *scales):
            t.view(torch.uint8).zero_()
        k, _ = fa.rope(k0, None, freqs, pos)
        q, _ = fa.rope(q0, None, freqs, qpos)
        fa.cache_append_fp8(k, v0, *pages, *scales, table, lens0, cu)
        q = q.view(B, Nq, Hq, d)
        o, lse = fa.decode_paged_fp8(q, *pages, *scales, table, lens0)
        t1, l1, free, n = fa.pages_fork([*pages, *scales], table, lens0, parent, ps)
        t2, live = fa.pages_compact([*pages, *scales], t1, l1, ps)
        o2, lse2 = fa.decode_paged_fp8(q, *pages, *scales, t2, l1)
        got = [x.clone() for x in (o, lse, t1, l1, free, n, t2, live, o2, lse2)]
        if first is None:
            first = got
        for a, b in zip(got, first):
            assert torch.equal(a.view(torch.uint8) if a.is_floating_point() else a,
                               b.view(torch.uint8) if b.is_floating_point() else b), turn
    assert fa.fa_last_device_error() == fa.FA_OK

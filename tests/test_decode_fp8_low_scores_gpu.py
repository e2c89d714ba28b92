"""Decode over the e4m3 cache where every score is far below 0, or every V block is zero: references are
set anywhere, from the first chunk on.  Against attention in 64 bits, with the tolerances of
test_cache_fp8_gpu.py."""
import math

import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa
from test_cache_fp8_gpu import _score_bound, check

pytestmark = pytest.mark.gpu
ROWS = pytest.mark.parametrize("Hq", [4, 16, 24, 40], ids=["4rows", "16rows", "24rows", "40rows"])


def _positive_k(seed, lens, d=128, ps=64, sb=32):
    rng = np.random.default_rng(seed)
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, 1, d, spread=0.5)
    return rng, kc & 0x7F, ks, vc, vs, table, sb


def _queries(rng, B, Nq, Hq, kc, ks, table, lens, sb, mean):
    """Negative elements; the mean score of a query over its sequence is -mean at scale 1."""
    q = -np.abs(rng.standard_normal((B, Nq, Hq, kc.shape[3]))) - 0.25
    for b in range(B):
        k = cache8.gather(kc, ks, table[b], lens[b], sb)[:, 0]
        q[b] *= mean / np.abs(q[b] @ k.mean(0))[..., None]
    return torch.from_numpy(q).cuda().bfloat16()


@ROWS
@pytest.mark.parametrize("mean", [100, 200, 1000])
@pytest.mark.parametrize("lens", [[1], [300, 129, 16], [20000]], ids=["one", "ragged", "cut"])
def test_scores_far_below_zero(lens, mean, Hq):
    rng, kc, ks, vc, vs, table, sb = _positive_k(6001, lens)
    q = _queries(rng, len(lens), 1, Hq, kc, ks, table, lens, sb, mean)
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1.0)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=1.0)
    check(o, lse, ref, q, (kc, ks, vc, vs, table, lens, sb, 1.0))


@ROWS
def test_a_low_chunk_before_ordinary_ones(Hq):
    """The first 128 rows, and every tenth chunk, score about -150, the others the opposite."""
    lens = [6000, 260]
    rng, kc, ks, vc, vs, table, sb = _positive_k(6002, lens)
    q = _queries(rng, 2, 1, Hq, kc, ks, table, lens, sb, 150)
    for b, n in enumerate(lens):
        j = np.arange(n)
        j = j[j // 128 % 10 != 0]
        kc[table[b, j // 64], j % 64] |= 0x80
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    ref = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1.0)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=1.0)
    check(o, lse, ref, q, (kc, ks, vc, vs, table, lens, sb, 1.0))


@ROWS
@pytest.mark.parametrize("mean", [30, 300])
@pytest.mark.parametrize("lens", [[33], [128, 500], [20000]], ids=["short", "ragged", "cut"])
def test_zero_v_with_low_scores(lens, mean, Hq):
    """Blocks of zeros have scale 0: o is 0 and lse is that of the scores."""
    rng, kc, ks, vc, vs, table, sb = _positive_k(6003, lens)
    q = _queries(rng, len(lens), 1, Hq, kc, ks, table, lens, sb, mean)
    for b, n in enumerate(lens):
        j = np.arange(n)
        vc[table[b, j // 64], j % 64] = 0
        vs[table[b, j // 64], :, j % 64 // sb] = 0.0
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    _, r_lse, _, _, t_abs = cache8.attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, lens, sb, 1.0)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=1.0)
    assert torch.all(o == 0)
    u = 0.0 if Hq <= 16 else _score_bound(q.double().cpu().numpy(), (kc, ks, vc, vs, table, lens, sb, 1.0))
    assert np.all(np.abs(lse.double().cpu().numpy() - r_lse) <= 2.0 ** -17 * (1 + t_abs + u))

"""Decode over the e4m3 cache where the V scales of one sequence lie far apart: every key keeps its
share of the softmax's sum, whatever its scale.

lse: 2^-17 (1 + t), as in test_cache_fp8_gpu.py.  o: half a bf16 step; the fp16 weights' 2^-11 and the
scores' 2^-17 (1 + t), relative; and 2^-25 of the largest weight, which is at least 1, for a code of at
most 448."""
import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa
from test_cache_fp8_gpu import _score_bound, _weight_max

pytestmark = pytest.mark.gpu


def _far_scales(lens, Hq, d, place, ps=32, sb=16):
    """place(block number, number of blocks) -> the scale's factor: 0 or an exponent of 2 as a float."""
    rng = np.random.default_rng(6101)
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, 1, d, spread=0.5)
    for b, n in enumerate(lens):
        blocks = (n + sb - 1) // sb
        for x in range(blocks):
            vs[table[b, x * sb // ps], :, x * sb % ps // sb] = place(x, blocks)
    q = torch.from_numpy(rng.standard_normal((len(lens), 1, Hq, d)) * 0.25).cuda().bfloat16()
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    q64 = q.double().cpu().numpy()
    r_o, r_lse, o_abs, _, t_abs = cache8.attend(q64, kc, ks, vc, vs, table, lens, sb, 1.0)
    o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5], scale=1.0)
    u = _score_bound(q64, (kc, ks, vc, vs, table, lens, sb, 1.0)) if Hq > 16 and d == 128 else 0.0
    assert np.all(np.abs(lse.double().cpu().numpy() - r_lse) <= 2.0 ** -17 * (1 + t_abs + u))
    top = _weight_max(q64, kc, ks, vs, table, lens, sb)
    tt = (t_abs + u).transpose(0, 2, 1)[..., None]
    tol = 2.0 ** -8 * np.abs(r_o) + (2.0 ** -11 + 2.0 ** -17 * (1 + tt)) * o_abs + max(lens) * 2.0 ** -25 * 448 * top
    assert np.all(np.abs(o.double().cpu().numpy() - r_o) <= tol)


@pytest.mark.parametrize("Hq,d", [(4, 128), (16, 128), (40, 128), (24, 64), (40, 64)])
@pytest.mark.parametrize("lens", [[256], [700, 90], [24000]], ids=["two chunks", "ragged", "cut"])
@pytest.mark.parametrize("way", ["up", "down", "64", "zeros first", "zeros last", "turns"])
def test_v_scales_far_apart(way, lens, Hq, d):
    place = {
        "up": lambda x, n: 2.0 ** (-90 if 2 * x < n else 90),
        "down": lambda x, n: 2.0 ** (90 if 2 * x < n else -90),
        "64": lambda x, n: 2.0 ** (-64 if 2 * x < n else 64),
        "zeros first": lambda x, n: 0.0 if 2 * x < n else 2.0 ** 60,
        "zeros last": lambda x, n: 2.0 ** 60 if 2 * x < n else 0.0,
        "turns": lambda x, n: 2.0 ** (-95 + 190 * x / max(n - 1, 1)) if n > 1 else 1.0,
    }[way]
    _far_scales(lens, Hq, d, lambda x, n: float(2.0 ** np.round(np.log2(place(x, n)))) if place(x, n) else 0.0)

"""NaN codes of V under finite scales, where several row groups of one unit read the same tile (d = 64, more
than 32 query rows): every query that attends to such a code gets NaN in its column, no other one does,
and a call repeats its bits."""
import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


def _nan_case(lens, Nq, Hq, d, spots, repeat, ps=32, sb=16):
    """spots: (sequence, token, column) of the NaN codes."""
    rng = np.random.default_rng(6301)
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, 1, d, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((len(lens), Nq, Hq, d))).cuda().bfloat16()
    clean = cache8.to_device(kc, ks, vc, vs, table, lens)
    o0, l0 = fa.decode_paged_fp8(q, clean[0], clean[2], clean[1], clean[3], clean[4], clean[5])
    assert not torch.isnan(o0).any()
    want = torch.zeros(o0.shape, dtype=torch.bool, device="cuda")
    for b, j, col in spots:
        vc[table[b, j // ps], j % ps, 0, col] = 0x7F if (j + col) % 2 else 0xFF
        want[b, max(0, j - (lens[b] - Nq)):, :, col] = True
    dev = cache8.to_device(kc, ks, vc, vs, table, lens)
    for turn in range(repeat):
        o, lse = fa.decode_paged_fp8(q, dev[0], dev[2], dev[1], dev[3], dev[4], dev[5])
        assert torch.equal(torch.isnan(o), want), turn
        assert torch.equal(lse, l0), turn
        if turn == 0:
            first = o[~want].clone()
            # a code of zero in its place changes other columns' bits nowhere
            cols = ~want.flatten(0, 2).any(0)
            assert torch.equal(o[..., cols], o0[..., cols])
        assert torch.equal(o[~want], first), turn
    assert fa.fa_last_device_error() == fa.FA_OK


@pytest.mark.parametrize("Hq", [33, 40, 48, 64])
def test_one_token_last_partial_tile(Hq):
    """Nq = 1: both row groups see all rows, and the last tile is partly past the end."""
    _nan_case([37, 153, 16, 530], 1, Hq, 64, [(0, 36, 0), (1, 150, 63), (1, 144, 17), (3, 529, 8), (3, 3, 30)], 100)


@pytest.mark.parametrize("Nq,Hq", [(3, 16), (4, 12), (8, 5), (2, 32), (40, 2)])
def test_new_tokens_that_see_it_and_that_do_not(Nq, Hq):
    """Codes in rows that some of the new tokens see: a group's tokens may see all, some or none of them."""
    lens = [Nq + 5, 200, 129]
    spots = [(b, lens[b] - 1 - k, c) for b, k, c in ((0, 0, 3), (0, 1, 44), (1, 1, 3), (2, 0, 63), (2, Nq - 1, 20),
                                                     (1, Nq // 2, 10))]
    _nan_case(lens, Nq, Hq, 64, spots, 100)


@pytest.mark.parametrize("Hq,d", [(4, 64), (12, 64), (24, 64), (8, 128), (16, 128), (24, 128), (64, 128)])
def test_the_other_kernels(Hq, d):
    _nan_case([37, 153, 16, 530], 1, Hq, d, [(0, 36, 0), (1, 150, 63), (1, 144, 17), (3, 529, 8), (3, 3, 30)], 5)
    _nan_case([39, 153], 3, Hq, d, [(0, 38, 1), (0, 37, 50), (1, 151, 50)], 5)

"""fa_pages_fork and fa_pages_compact against a plain model on the host: tables, lengths, free
lists and every byte of the pools, exactly."""
import numpy as np
import pytest
import torch

import cache8
from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


def fork_model(table, lens, parent, ps, P):
    R, M = len(parent), table.shape[1]
    out, n_out = np.full((R, M), -1, np.int32), np.zeros(R, np.int32)
    full, owner, tails = set(), {}, {}
    for i, b in enumerate(parent):
        if b < 0:
            continue
        n_out[i] = lens[b]
        k = -(-lens[b] // ps)
        out[i, :k] = table[b, :k]
        full.update(table[b, :lens[b] // ps].tolist())
        if lens[b] % ps:
            tails[i] = int(table[b, lens[b] // ps])
            owner.setdefault(tails[i], i)
    free = [p for p in range(P) if p not in full and p not in owner]
    moves = []
    for i, page in tails.items():
        if page in full or owner[page] != i:
            if not free:
                out[i], n_out[i] = -1, 0
                continue
            to = free.pop(0)
            moves.append((page, to))
            out[i, lens[parent[i]] // ps] = to
    return out, n_out, free, moves


def compact_model(table, lens, ps, P):
    M = table.shape[1]
    held = np.arange(M)[None] < -(-lens // ps)[:, None]
    live = sorted(set(table[held].tolist()))
    n = len(live)
    holes = [p for p in range(n) if p not in set(live)]
    to = dict(zip([p for p in live if p >= n], holes))
    out = np.where(held, np.vectorize(lambda p: to.get(p, p))(table), -1).astype(np.int32)
    return out, n, list(to.items())


def pools_of(rng, P, kinds):
    return [torch.from_numpy(rng.integers(0, 256, (P, *k), dtype=np.uint8)).cuda() for k in kinds]


def layout(rng, lens, ps, spare, M=None):
    need = -(-np.array(lens) // ps)
    P = max(1, int(need.sum()) + spare)
    order = rng.permutation(P)
    table = np.full((len(lens), M or max(1, int(need.max()))), -5, np.int32)  # unused entries: anything
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, P


def check_pools(pools, before, moves):
    for p, b in zip(pools, before):
        want = b.clone()
        for s, d in moves:
            want[d] = b[s]
        assert torch.equal(p, want)


dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731

FORKS = [
    # lens, parents, page_size, spare pages, pool page shapes
    ([5], [0], 16, 0, [(16, 3)]),
    ([5], [0, 0, 0], 16, 2, [(16, 64), (1,)]),
    ([16, 0, 33], [2, 2, 1, -1, 0, 0], 16, 40, [(640,), (7,), (12,)]),
    ([100, 200, 300], [], 32, 3, [(16,)]),
    ([1, 64, 65, 127], [3, 1, 3, 0, 2, 3, 0], 64, 9, [(64, 33), (4,)]),
    ([1000] * 7 + [17], list(range(8)) * 9, 16, 70, [(2048,)]),
    ([300, 77, 128], [0, 0, 1, 1, 2, 2], 128, 4, [(128, 321), (40016,), (5000,)]),
    ([31] * 300, [i // 4 for i in range(1200)], 8, 1500, [(48,), (20,)]),
]


@pytest.mark.parametrize("case", FORKS, ids=[f"{len(c[0])}to{len(c[1])}_p{c[2]}" for c in FORKS])
def test_fork_matches_model(case):
    lens, parent, ps, spare, kinds = case
    rng = np.random.default_rng(6001)
    table, P = layout(rng, lens, ps, spare)
    pools = pools_of(rng, P, kinds)
    before = [p.clone() for p in pools]
    t, n, free, moves = fork_model(table, np.array(lens), parent, ps, P)
    for _ in range(2):  # the same call again: nothing it reads has changed
        gt, gn, gf, gc = fa.pages_fork(pools, dev(table), dev(lens), dev(np.array(parent, np.int32)), ps)
        assert np.array_equal(gt.cpu().numpy(), t) and np.array_equal(gn.cpu().numpy(), n)
        assert int(gc) == len(free)
        assert gf.cpu().tolist() == free + [-1] * (P - len(free))
        check_pools(pools, before, moves)
    assert fa.fa_last_device_error() == fa.FA_OK


def test_fork_of_a_shortened_sequence_copies_a_shared_page():
    """Two sequences share a full page; one is cut back into it: its heir must not write there."""
    rng = np.random.default_rng(6002)
    table, ps, P = np.array([[3, 1], [3, 2]], np.int32), 16, 6
    lens, parent = np.array([32, 9]), [0, 1, 1]
    pools = pools_of(rng, P, [(16, 5)])
    before = [p.clone() for p in pools]
    gt, gn, gf, gc = fa.pages_fork(pools, dev(table), dev(lens), dev(parent), ps)
    assert gt.cpu().tolist() == [[3, 1], [0, -1], [2, -1]]
    assert gn.cpu().tolist() == [32, 9, 9] and gf.cpu().tolist()[:int(gc)] == [4, 5]
    check_pools(pools, before, [(3, 0), (3, 2)])


def test_fork_without_enough_pages_empties_the_last_heirs():
    rng = np.random.default_rng(6003)
    table, P = layout(rng, [5, 20], 16, 1)
    pools = pools_of(rng, P, [(32,)])
    parent = [0, 0, 0, 1]
    t, n, free, moves = fork_model(table, np.array([5, 20]), parent, 16, P)
    gt, gn, gf, gc = fa.pages_fork(pools, dev(table), dev([5, 20]), dev(parent), 16)
    assert fa.fa_last_device_error() == fa.FA_ERR_INVALID_ARG
    assert np.array_equal(gt.cpu().numpy(), t) and gn.cpu().tolist() == n.tolist() == [5, 5, 0, 20]
    assert int(gc) == 0 and len(moves) == 1


def test_pages_record_and_skip_bad_entries():
    rng = np.random.default_rng(6004)
    pools = pools_of(rng, 8, [(16,)])
    before = [p.clone() for p in pools]
    table = np.array([[1, 99], [2, 3], [-4, 0]], np.int32)
    gt, gn, gf, gc = fa.pages_fork(pools, dev(table), dev([20, 1000, 5]), dev([0, 0, 1, 7, 2]), 16)
    assert fa.fa_last_device_error() == fa.FA_ERR_INVALID_ARG
    assert gt.cpu().tolist() == [[1, 99], [1, 99], [-1, -1], [-1, -1], [-4, -1]]
    assert gn.cpu().tolist() == [20, 20, 0, 0, 5]
    check_pools(pools, before, [])
    gt, gl = fa.pages_compact(pools, dev(table), dev([20, -3, 5]), 16)
    assert fa.fa_last_device_error() == fa.FA_ERR_INVALID_ARG
    assert gt.cpu().tolist() == [[0, 99], [-1, -1], [-4, -1]] and int(gl) == 1
    check_pools(pools, before, [(1, 0)])
    assert fa.fa_last_device_error() == fa.FA_OK


COMPACTS = [
    ([5], 16, 0, [(16,)]),
    ([0, 0], 16, 5, [(16,)]),
    ([100, 0, 33, 1], 16, 30, [(640,), (7,), (12,)]),
    ([64] * 40, 64, 40, [(4096,)]),
    ([700, 130, 1], 128, 9, [(128, 321), (40016,), (16384,)]),
    ([3000, 17, 900], 16, 2000, [(48,), (20,)]),
    ([5] * 2000, 8, 2100, [(4,)]),
]


@pytest.mark.parametrize("case", COMPACTS, ids=[f"{len(c[0])}seq_p{c[1]}_{c[2]}spare" for c in COMPACTS])
def test_compact_matches_model(case):
    lens, ps, spare, kinds = case
    rng = np.random.default_rng(6005)
    table, P = layout(rng, lens, ps, spare, M=int(max(1, -(-max(lens) // ps))) + 1)
    pools = pools_of(rng, P, kinds)
    before = [p.clone() for p in pools]
    t, n, moves = compact_model(table, np.array(lens), ps, P)
    for _ in range(2):
        gt, gl = fa.pages_compact(pools, dev(table), dev(lens), ps)
        assert np.array_equal(gt.cpu().numpy(), t) and int(gl) == n
        check_pools(pools, before, moves)
    # compacting what is compact moves nothing
    t2, l2 = fa.pages_compact(pools, gt, dev(lens), ps)
    assert torch.equal(t2, gt) and int(l2) == n
    check_pools(pools, before, moves)
    assert fa.fa_last_device_error() == fa.FA_OK


def test_many_pools_and_unaligned_ones():
    """More pools than one launch takes, some off a 16-byte boundary."""
    rng = np.random.default_rng(6006)
    lens, ps = [40, 3, 25], 16
    table, P = layout(rng, lens, ps, 8)
    parent = [0, 0, 1, 1, 2, 2]
    pools = []
    for j in range(300):
        size = (33, 32, 4096, 20000)[j % 4]  # two of them large enough for bulk copies
        raw = torch.from_numpy(rng.integers(0, 256, 1 + P * size, dtype=np.uint8)).cuda()
        pools.append(raw[j % 5 == 0:][:P * size].view(P, size))
    before = [p.clone() for p in pools]
    t, n, free, moves = fork_model(table, np.array(lens), parent, ps, P)
    gt, *_ = fa.pages_fork(pools, dev(table), dev(lens), dev(parent), ps)
    assert np.array_equal(gt.cpu().numpy(), t)
    check_pools(pools, before, moves)


def test_forked_sequences_decode_and_grow_apart():
    """Fork, append a different token to each heir, compact, decode: every heir reads its parent's
    rows and its own; also over bf16 pages with fa_decode_paged."""
    rng = np.random.default_rng(6007)
    lens, parent, ps, sb, H, d = [37, 16], [0, 0, 1, 0], 16, 16, 1, 64
    kc, ks, vc, vs, table = cache8.build(rng, lens, ps, sb, H, d, extra=9)
    a = cache8.to_device(kc, ks, vc, vs, table, lens)
    b_pages = torch.from_numpy(rng.standard_normal((kc.shape[0], ps, H, d))).cuda().bfloat16()
    pools = [a[0], a[1], a[2], a[3], b_pages]
    q = torch.from_numpy(rng.standard_normal((4, 2, d))).cuda().bfloat16()
    par = torch.tensor(parent, device="cuda")
    o_b, _ = fa.decode_paged(q, b_pages, b_pages, a[4][par].contiguous(), a[5][par].contiguous())
    o_8, _ = fa.decode_paged_fp8(q, a[0], a[2], a[1], a[3], a[4][par].contiguous(), a[5][par].contiguous())
    t, n, free, cnt = fa.pages_fork(pools, a[4], a[5], dev(parent), ps)
    got_b, _ = fa.decode_paged(q, b_pages, b_pages, t, n)
    got_8, _ = fa.decode_paged_fp8(q, a[0], a[2], a[1], a[3], t, n)
    assert torch.equal(o_b, got_b) and torch.equal(o_8, got_8)
    # sequence 2 has a full last page: it takes a free page for its next row
    t[2, 1] = free[0]
    n += 1
    new = torch.from_numpy(rng.standard_normal((4, H, d))).cuda().bfloat16()
    fa.cache_append_fp8(new, new, a[0], a[2], a[1], a[3], t, n)
    o1, l1 = fa.decode_paged_fp8(q, a[0], a[2], a[1], a[3], t, n)
    host = [a[0].view(torch.uint8).cpu().numpy(), a[1].double().cpu().numpy(), t.cpu().numpy()]
    for i, b in enumerate(parent):
        rows = cache8.gather(host[0], host[1], host[2][i], int(n[i]), sb)
        was = cache8.gather(kc, ks, table[b], lens[b], sb)
        grew = rows[:lens[b]] != was  # only a rescaled last block may differ, below its normal range
        assert not grew[:lens[b] // sb * sb].any()
        x = new[i].double().cpu().numpy()
        s = host[1][host[2][i, lens[b] // ps], :, 0]
        assert np.all(np.abs(rows[-1] - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s[:, None])
    t2, live = fa.pages_compact(pools, t, n, ps)
    o2, l2 = fa.decode_paged_fp8(q, a[0], a[2], a[1], a[3], t2, n)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert int(t2.max()) < int(live)
    assert fa.fa_last_device_error() == fa.FA_OK

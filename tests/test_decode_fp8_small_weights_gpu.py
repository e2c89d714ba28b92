"""Decode over the e4m3 cache for more than 16 query rows where one key outweighs every other one by far,
and the others together still count: nothing of their weights is lost.

Every key but one has score 0 (K = 0), the one has the head's gap: o = (e^gap v_0 + sum v_j) / (e^gap +
n - 1) in 64 bits.  Tolerance, relative to sum p|v|: half a bf16 step of o, 2^-8; the fp16 weights, 2^-11,
and half a step of 2^-24 where they are small and the largest is at least 2^8, n 2^-33 of that; 2^-17 (1 +
gap) for scores and exponentials; sums of products over a run of 32K keys, 2048 additions that drop less
than 2^-22 each, 2^-11 (and runs are added in fp32); and the fp32 sum of p by 128 threads: of n / 128
additions in turn, each may be off by 2^-24 of the sum so far, n 2^-31 in all (a million keys: 4.9e-4,
where lse was off by 3.3e-4)."""
import pytest
import torch

from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


def _run(n, Hq, gaps, at, d=128, B=300, ps=256, sb=256):
    """B sequences over the same pages: more than there are CTAs, so that some CTA takes one whole."""
    g = torch.Generator(device="cuda").manual_seed(6201)
    P = (n + ps - 1) // ps
    kc = torch.zeros(P, ps, 1, d, dtype=torch.uint8, device="cuda")
    kc.view(-1, d)[at] = 0x38  # 1.0
    # V about 1: codes of 0.5 .. 1.875, so that what is lost shows
    vc = torch.randint(0x30, 0x40, (P, ps, 1, d), generator=g, device="cuda", dtype=torch.uint8)
    one = torch.ones(P, 1, ps // sb, device="cuda")
    table = torch.randperm(P, generator=g, device="cuda").int().view(1, P)
    back = torch.empty(P, dtype=torch.int64, device="cuda")
    back[table[0].long()] = torch.arange(P, device="cuda")
    kc, vc = kc[back].contiguous(), vc[back].contiguous()  # page table[t] holds tokens t ps ..
    gap = torch.tensor([gaps[h % len(gaps)] for h in range(Hq)], dtype=torch.float64, device="cuda")
    q = (gap[:, None] / d).expand(Hq, d).bfloat16()
    gap = q.double().sum(1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, lse = fa.decode_paged_fp8(q.expand(B, Hq, d).contiguous(), kc.view(torch.float8_e4m3fn),
                                 vc.view(torch.float8_e4m3fn), one, one, table.expand(B, P).contiguous(), lens,
                                 scale=1.0)
    v = vc[table[0].long()].view(-1, d)[:n].view(torch.float8_e4m3fn)
    total, v0 = torch.zeros(d, dtype=torch.float64, device="cuda"), v[at].double()
    for part in v.split(1 << 18):
        total += part.double().sum(0)
    w = gap.exp()[:, None]
    ref = (w * v0 + total - v0) / (w + n - 1)
    z = 1 + (n - 1) / w  # sum of p over the largest
    added = n * 2.0 ** -31
    tol = (2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -17 * (1 + gap[:, None]) + added) * ref + n * 2.0 ** -33 * 1.875 / z
    worst = ((o.double() - ref).abs() / tol).max()
    assert worst <= 1, float(worst)
    r_lse = gap + torch.log1p((n - 1) / w[:, 0])
    assert torch.all((lse.double() - r_lse).abs() <= 2.0 ** -17 * (1 + 2 * gap) + added)


@pytest.mark.parametrize("at", [0, 1000, 32000])
@pytest.mark.parametrize("Hq", [24, 40, 64])
def test_one_key_far_above_many(Hq, at):
    _run(32768 + 77, Hq, [9.0, 10.0, 11.0, 11.5, 12.0, 13.0], at)


@pytest.mark.parametrize("n,at", [(32768, 5), (32768 + 128, 32768), (70000, 40000), (131072 + 1, 131072)])
def test_sums_in_runs(n, at):
    """The sums of 32K keys are moved on; the key that outweighs the others comes before or after."""
    _run(n, 33, [0.0, 2.0, 9.0, 11.0, 12.0, 13.0], at)


def test_one_key_far_above_a_million():
    _run((1 << 20) + 5, 20, [12.0, 13.0, 14.0, 15.0], 0)

"""Sines and cosines of fa_rope in fp32, read off unit vectors: off by at most one unit in the last place of
a value below 1 (sincospif) and half a unit for putting back what the angle's rounding took, 1.5 * 2^-24;
an angle of half a turn and more rounded to fp32 alone would add up to pi 2^-25.  The angle itself is off
by three fp64 roundings in the kernel (times the frequency, 1 / 2 pi and their product) and one here:
4 * 2^-53 of it."""
import pytest
import torch

from exact_io_aware_97_b200 import binding as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 50])
@pytest.mark.parametrize("far", [1, 1 << 20, 1 << 30])
def test_sines_and_cosines_of_fp32(far, rot, interleaved):
    n, d = 20000, 64
    freqs = fa.rope_frequencies(rot, 10000.0)
    pos = torch.arange(-n // 2, n // 2, device="cuda").int() * (far if far == 1 else far // n)
    x = torch.zeros(n, 1, d, device="cuda")
    a = torch.arange(rot // 2, device="cuda")
    a, b = (2 * a, 2 * a + 1) if interleaved else (a, a + rot // 2)
    x[:, 0, a] = 1.0
    y, _ = fa.rope(x, None, freqs, pos, interleaved)
    angle = pos.double()[:, None] * freqs
    tol = 1.5 * 2.0 ** -24 + 4 * 2.0 ** -53 * angle.abs()
    assert torch.all((y[:, 0, a].double() - torch.cos(angle)).abs() <= tol)
    assert torch.all((y[:, 0, b].double() - torch.sin(angle)).abs() <= tol)

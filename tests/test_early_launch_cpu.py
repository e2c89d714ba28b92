"""Kernels that may be launched while the stream's last kernel ends exist while that one still writes
what they read: each of them waits before it touches memory, and none reads through the read-only path
(__ldg, ld.global.nc), which is for memory that nothing writes while the kernel exists."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_97_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


EARLY = sorted(f for f in os.listdir(CSRC) if f.endswith(".cuh") and f != "fa_device.cuh" and "grid_wait()" in _code(f))


def test_the_early_kernels_are_found():
    assert {"fa_rope.cuh", "fa_cache.cuh", "fa_decode_fp8.cuh", "fa_decode_fp8_narrow.cuh", "fa_decode_fp8_tc.cuh",
            "fa_pages.cuh"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_no_read_only_loads(name):
    assert not re.search(r"__ldg\s*\(|ld\.global[.\w]*\.nc|__restrict__", _code(name))


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits(name):
    kernels = _code(name).split("__global__")[1:]
    assert kernels and all("grid_wait();" in k for k in kernels)

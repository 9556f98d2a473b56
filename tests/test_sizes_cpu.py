"""Sizes whose products leave 64 bits are refused like other sizes past a launch (no GPU)."""
import ctypes

import pytest

from semi_markov_crf_zero_amd import encoder

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("name", ["semicrf_delta_workspace_size", "semicrf_linattn_workspace_size"])
@pytest.mark.parametrize("B,T,H", [(MOST, 1, MOST), (MOST, 5, MOST), (MOST, 1 << 30, MOST), (1 << 30, 1, 1 << 30),
                                   (1 << 28, 32, 1 << 27), (1 << 30, 1 << 30, 1 << 16), (MOST, 1, 2)])
def test_products_past_64_bits(name, B, T, H):
    lib, n = encoder.load(), ctypes.c_size_t(0)
    s = encoder._LinattnShape(B, T, H, H, H, H, 8, 8, 1, 1.0)
    for way in (0, 1):
        assert getattr(lib, name)(ctypes.byref(s), way, ctypes.byref(n)) == 2


def test_the_largest_that_a_launch_holds():
    lib, n = encoder.load(), ctypes.c_size_t(0)
    size = lambda B, T, H: lib.semicrf_delta_workspace_size(  # noqa: E731
        ctypes.byref(encoder._LinattnShape(B, T, H, H, H, H, 8, 8, 1, 1.0)), 0, ctypes.byref(n))
    for B, T, H in (((1 << 23) - 1, 1, 1), ((1 << 22) - 1, 33, 1), (1, 1 << 28, 1)):
        want = 0 if B * H * -(-T // 32) < 1 << 23 else 2
        assert size(B, T, H) == want, (B, T, H)
    assert size(1 << 23, 1, 1) == 2 and size(1, 1 << 28, 1) == 2 and size(1, (1 << 28) - 32, 1) == 0

"""The attention kernels' division by multiplication, on the CPU."""

import numpy as np


def test_division_by_multiplication():
    """floor(x m / 2^(31+L)) with m = floor(2^(31+L) / d) + 1, 2^L <= d < 2^(L+1), is
    floor(x / d) for x < 2^30, d <= 1024: at every multiple's two sides for the small
    and the large multiples, and in between at random."""
    rng = np.random.default_rng(0)
    top = 2 ** 30 - 1
    for d in range(1, 1025):
        L = d.bit_length() - 1
        m = 2 ** (31 + L) // d + 1
        assert m < 2 ** 32
        q = np.concatenate([np.arange(1, 200), top // d - np.arange(200), rng.integers(1, top // d + 1, 200)])
        x = np.concatenate([q * d - 1, q * d, [0, top]])
        x = x[(x >= 0) & (x <= top)].astype(np.uint64)
        got = (x * np.uint64(m)) >> np.uint64(31 + L)
        assert (got == x // np.uint64(d)).all()

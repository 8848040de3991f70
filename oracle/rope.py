"""Oracle: rotary positions.

TEST INFRASTRUCTURE ONLY (see the package docstring).  `rotate64` is the formula in
fp64; `rotate32` takes the steps that include/awq355.h gives (cosines and sines
rounded to fp32, fp32 products and sums), which a cache's codes depend on.
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(R, base=10000.0, scaling="none", s=1.0, L=0.0, low=0.0, high=0.0):
    """(inv_freq [R/2], attention factor), pair by pair."""
    out = []
    for j in range(R // 2):
        f = base ** (-2.0 * j / R)
        if scaling == "linear":
            f /= s
        elif scaling == "ntk":
            f = (base * s ** (R / (R - 2.0))) ** (-2.0 * j / R)
        elif scaling == "yarn":
            pair = lambda n: R * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
            a, b = max(math.floor(pair(high or 32.0)), 0), min(math.ceil(pair(low or 1.0)), R - 1)
            m = min(max((j - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f / s * m + f * (1 - m)
        elif scaling == "bands":
            turns, lo, hi = L * f / (2 * math.pi), low or 1.0, high or 4.0
            m = min(max((turns - lo) / (hi - lo), 0.0), 1.0)
            f = f if turns > hi else f / s if turns < lo else (1 - m) / s * f + m * f
        out.append(f)
    return np.array(out), (0.1 * math.log(s) + 1 if scaling == "yarn" and s > 1 else 1.0)


def _channels(R, interleaved):
    j = np.arange(R // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)


def rotate64(x, pos, inv, factor=1.0, interleaved=False, inverse=False):
    """x fp64 [T][heads][D] rotated; and per element |own c| + |partner s|, which errors scale with."""
    x = np.asarray(x, np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    a, b = _channels(2 * len(inv), interleaved)
    ang = np.asarray(pos, np.float64)[:, None] * inv
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None] * (-1 if inverse else 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def rotate32(x, pos, inv, factor=1.0, interleaved=False):
    """x fp32 [T][heads][D] rotated in the documented fp32 steps."""
    x = np.asarray(x, np.float32)
    y = x.copy()
    a, b = _channels(2 * len(inv), interleaved)
    ang = np.asarray(pos, np.float64)[:, None] * inv
    c, s = (factor * np.cos(ang)).astype(np.float32)[:, None], (factor * np.sin(ang)).astype(np.float32)[:, None]
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y

"""fp64 per-head RMS norm and rotary positions, value by value.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Norm: x / sqrt(mean(x^2) + eps) * w over a head's values.  Rotation: pair j of a
head's first r values is turned by position * f_j; the pairs are (j, j + r/2),
or (2j, 2j + 1) when interleaved; the other values stay."""

from __future__ import annotations

import math

import numpy as np

from .attention import f64


def norm_ref(x, weight, eps: float) -> np.ndarray:
    x = f64(x)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(weight)


def rotate_ref(x, positions, inv_freq, interleaved: bool, scale: float = 1.0) -> np.ndarray:
    """x [T, H, d] -> the same, turned; angles with Python's own pi-free
    cos / sin of the fp64 product position * frequency."""
    x = f64(x)
    out = x.copy()
    half = len(inv_freq)
    for t, p in enumerate(np.asarray(positions).tolist()):
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            w = p * float(inv_freq[j])
            c, s = scale * math.cos(w), scale * math.sin(w)
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out

"""fp64 oracle of the norms of queries and keys with the position rotation
(include/qkrope.h), pair by pair in plain numpy. Test infrastructure only.

    n = x / sqrt(mean(x^2) + eps) * weight;  y = n, pair j of it turned by position * freq_j
"""
from __future__ import annotations

import numpy as np


def _turned(x, angle, interleaved):
    """x [...][D] with pair j turned by angle [...][half] (broadcast over heads)."""
    half = angle.shape[-1]
    y = x.copy()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, half + j)
        c, s = np.cos(angle[..., j]), np.sin(angle[..., j])
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def _angles(positions, freq):
    # (positions up to 2^31 times frequencies: to 2^-53 of the product)
    return (positions.astype(np.float64)[..., None] * freq)[..., None, :]


def forward(x, weight, freq, positions, *, interleaved=False, eps=1e-6):
    """x [...][H][D], positions [...]."""
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turned(x / rms * weight, _angles(positions, freq), interleaved)


def backward(x, weight, freq, positions, dy, *, interleaved=False, eps=1e-6):
    """(dx, dweight) of sum <dy, y>."""
    d = _turned(dy, -_angles(positions, freq), interleaved)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    t = d * weight
    dx = t / rms - x * (t * x).mean(-1, keepdims=True) / rms ** 3
    return dx, (d * x / rms).reshape(-1, x.shape[-1]).sum(0)

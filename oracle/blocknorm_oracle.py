"""fp64 oracle of the block norms (include/blocknorm.h) in plain numpy. Test
infrastructure only."""
from __future__ import annotations

import numpy as np


def add(x, residual, weight, scale=None, *, eps=1e-6):
    """(h, n) with h = residual + scale x, n = h / rms(h) weight; x None: h = residual."""
    h = residual if x is None else residual + (x if scale is None else scale * x)
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight


def add_grad(x, residual, weight, dn, dh=None, scale=None, *, eps=1e-6):
    h, _ = add(x, residual, weight, scale, eps=eps)
    D = h.shape[-1]
    rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    t = dn * weight
    d = t / rms - h * (t * h).sum(-1, keepdims=True) / (D * rms ** 3)
    if dh is not None:
        d = d + dh
    rows = tuple(range(h.ndim - 1))
    out = {"dresidual": d, "dweight": (dn * h / rms).sum(rows)}
    if x is not None:
        out["dx"] = d if scale is None else scale * d
        if scale is not None:
            out["dscale"] = (d * x).sum(rows)
    return out


def _gate(z):
    s = 1 / (1 + np.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def gated(o, z, weight, *, eps=1e-6):
    return o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * weight * _gate(z)[0]


def gated_grad(o, z, weight, dy, *, eps=1e-6):
    D = o.shape[-1]
    rms = np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    gate, slope = _gate(z)
    t = dy * gate * weight
    rows = tuple(range(o.ndim - 1))
    return {"do": t / rms - o * (t * o).sum(-1, keepdims=True) / (D * rms ** 3), "dz": dy * o / rms * weight * slope,
            "dweight": (dy * gate * o / rms).sum(rows)}

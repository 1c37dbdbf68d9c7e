"""fp64 oracle of the per-head norm with the position rotation (test
infrastructure only, like the rest of this package)."""
from __future__ import annotations

import numpy as np


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _rotate(u, cos, sin, positions, interleaved, sign):
    """Every pair (a, b) of the first rot elements of u [T, H, d] turned by
    sign times the angle of the token's position."""
    c, s = (np.asarray(t, dtype=np.float64)[positions][:, None, :] for t in (cos, sin))
    a, b = _pairs(2 * c.shape[-1], interleaved)
    y = np.array(u, dtype=np.float64)
    y[..., a] = u[..., a] * c - sign * u[..., b] * s
    y[..., b] = u[..., b] * c + sign * u[..., a] * s
    return y


def norm_rope_forward(x, w, cos, sin, positions, eps, interleaved):
    """x [T, H, d], w [d], tables [max_pos, rot / 2], positions [T]."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return _rotate(x * r * w, cos, sin, positions, interleaved, 1.0)


def norm_rope_backward(x, w, cos, sin, positions, eps, interleaved, dy):
    """(dx, dw) of sum(norm_rope_forward * dy), and the sums of the magnitudes
    of the terms of dw (what its rounding errors scale with)."""
    x, w, dy = (np.asarray(t, dtype=np.float64) for t in (x, w, dy))
    r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r
    du = _rotate(dy, cos, sin, positions, interleaved, -1.0)
    dn = du * w
    dx = r * (dn - n * np.mean(dn * n, axis=-1, keepdims=True))
    return dx, np.sum(du * n, axis=(0, 1)), np.sum(np.abs(du * n), axis=(0, 1))

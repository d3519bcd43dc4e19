"""The residual RMS norm and gradient clipping in fp64 -- TEST INFRASTRUCTURE ONLY."""
from __future__ import annotations

import numpy as np

from .balance import _rows


def forward(s, weight, eps):
    """y of the rounded sum s [T, H]."""
    s = _rows(s)
    return np.stack([row / np.sqrt((row * row).mean() + eps) for row in s]) * _rows(weight)


def backward(dy, s, weight, eps, ds=None):
    """dx, dweight, and bounds on what their terms sum to in magnitude, through each row's Jacobian
    d y_i / d s_j = w_i (delta_ij r - s_i s_j r^3 / H)."""
    dy, s, w = _rows(dy), _rows(s), _rows(weight)
    T, H = s.shape
    dx, mag = np.zeros((T, H)), np.zeros((T, H))
    dw, wmag = np.zeros(H), np.zeros(H)
    for t in range(T):
        r = 1.0 / np.sqrt((s[t] * s[t]).mean() + eps)
        g = dy[t] * w
        dx[t] = r * g - s[t] * (r ** 3 / H) * (g @ s[t])
        mag[t] = r * np.abs(g) + np.abs(s[t]) * (r ** 3 / H) * (np.abs(g) @ np.abs(s[t]))
        dw += dy[t] * s[t] * r
        wmag += np.abs(dy[t] * s[t] * r)
    if ds is not None:
        dx += _rows(ds)
        mag += np.abs(_rows(ds))
    return dx, dw, mag, wmag


def clip(grads, max_norm, sumsq=None):
    """(norm, clipped gradients)."""
    g = [np.asarray(x, dtype=np.float64) for x in grads]
    if sumsq is None:
        sumsq = sum(float((x * x).sum()) for x in g)
    norm = float(np.sqrt(sumsq))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [x * c for x in g]

"""Routing by scores with a bias and groups, and its gradient, in fp64 -- TEST INFRASTRUCTURE ONLY.

Loops over tokens and sorts of Python tuples, apart from the kernels' networks: an order is (value
descending with NaN first, id ascending).  Without a bias experts (and groups of one best) go by their logits, whose order
is that of the scores as real numbers; else scores are compared as fp64 values.
"""
from __future__ import annotations

import math

import numpy as np

from .balance import _rows


def scores(lg: np.ndarray, score: str) -> np.ndarray:
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-lg))
        out = np.zeros_like(lg)
        for t, row in enumerate(lg):
            m = row.max()
            if m == -np.inf:
                continue
            e = np.exp(row - m)
            out[t] = e / e.sum()
        return out


def _order(values):
    """Ids by value descending (NaN first), then id."""
    return sorted(range(len(values)), key=lambda i: (0 if math.isnan(values[i]) else 1,
                                                     0.0 if math.isnan(values[i]) else -values[i], i))


def forward(logits, k, bias=None, score="sigmoid", groups=1, topk_groups=None, group_best=1, renormalize=True,
            scale=1.0, mask=None):
    """(idx int32 [T, k], prob [T, k], counts int32 [E])."""
    lg = _rows(logits)
    T, E = lg.shape
    n = E // groups
    topk_groups = groups if topk_groups is None else topk_groups
    s = scores(lg, score)
    c = s + (0.0 if bias is None else _rows(bias))
    c = np.where(lg == -np.inf, -np.inf, c)
    idx, prob = np.zeros((T, k), dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        v = (lg if bias is None else c)[t].copy()
        if groups > 1:
            sums = []
            for g in range(groups):
                part = (v if group_best == 1 else c[t])[g * n:(g + 1) * n]
                best = [part[i] for i in _order(part)[:group_best]]
                sums.append(best[0] + best[1] if group_best == 2 else best[0])
            for g in _order(sums)[topk_groups:]:
                v[g * n:(g + 1) * n] = -np.inf
        ids = _order(v)[:k]
        w = np.array([0.0 if v[i] == -np.inf else s[t, i] for i in ids])
        if renormalize:
            w = w / w.sum() if w.sum() != 0 else np.zeros(k)
        idx[t], prob[t] = ids, w * scale
    live = idx if mask is None else idx[np.asarray(mask).astype(bool)]
    return idx, prob, np.bincount(live.reshape(-1), minlength=E).astype(np.int32)


def weights(lg, idx, score, renormalize, scale):
    """The weights at fixed ids: what the gradient differentiates."""
    s = np.take_along_axis(scores(_rows(lg), score), np.asarray(idx, dtype=np.int64), axis=1)
    return scale * (s / s.sum(axis=1, keepdims=True) if renormalize else s)


def backward(logits, idx, prob, dprob, score="sigmoid", renormalize=True, scale=1.0):
    """dlogits [T, E] from the weights given, and a bound on what its terms sum to in magnitude."""
    lg = _rows(logits)
    T, E = lg.shape
    s = scores(lg, score)
    w, g = np.asarray(prob, dtype=np.float64), np.asarray(dprob, dtype=np.float64)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        dot, adot = float(w[t] @ g[t]), float(np.abs(w[t]) @ np.abs(g[t]))
        for j, e in enumerate(np.asarray(idx[t])):
            if not 0 <= e < E:
                continue
            with np.errstate(over="ignore"):
                slope = 1.0 / (1.0 + np.exp(lg[t, e])) if score == "sigmoid" else 1.0
            d[t, e] += slope * w[t, j] * (g[t, j] - (dot / scale if renormalize else 0.0))
            mag[t, e] += abs(slope * w[t, j]) * (abs(g[t, j]) + (adot / scale if renormalize else 0.0))
        if score == "softmax" and not renormalize:
            d[t] -= s[t] * dot
            mag[t] += s[t] * adot
    return d, mag

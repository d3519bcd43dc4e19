"""The training router's losses and gradients in fp64 -- TEST INFRASTRUCTURE ONLY.

Routing as oracle/router.py; with p = softmax(l) over all E experts, lse = log sum exp l, the n tokens
that count (not masked, and with a logit above -inf) and C_e how many of their slots went to e:

    L_b = E / (k n^2) sum_e C_e sum_t p[t, e]        L_z = 1/n sum_t lse_t^2

The counts are constants of L_b.  Written as loops over tokens, apart from the kernels' algebra: the
gradient goes through the softmax's Jacobian row by row.
"""
from __future__ import annotations

import numpy as np


def _rows(logits):
    if hasattr(logits, "detach"):
        import torch
        return logits.detach().to("cpu", torch.float64).numpy()
    return np.asarray(logits, dtype=np.float64)


def counting(logits, mask=None) -> np.ndarray:
    """Which tokens count."""
    lg = _rows(logits)
    live = lg.max(axis=1) > -np.inf
    return live if mask is None else live & np.asarray(mask).astype(bool)


def softmax_rows(lg):
    """(p, lse) of every row; a row without a logit above -inf gives zeros and 0."""
    p = np.zeros_like(lg)
    lse = np.zeros(lg.shape[0])
    for t, row in enumerate(lg):
        m = row.max()
        if m == -np.inf:
            continue
        e = np.exp(row - m)
        p[t] = e / e.sum()
        lse[t] = m + np.log(e.sum())
    return p, lse


def forward(logits, k: int, mask=None):
    """(idx int32 [T, k], prob [T, k], counts int32 [E], losses [2])."""
    lg = _rows(logits)
    T, E = lg.shape
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    prob = np.zeros((T, k))
    for t in range(T):
        v = lg[t, idx[t]]
        if v[0] == -np.inf:
            continue
        w = np.exp(v - v[0])
        prob[t] = w / w.sum()
    c = counting(lg, mask)
    p, lse = softmax_rows(lg)
    counts = np.bincount(idx[c].reshape(-1), minlength=E).astype(np.int32)
    return idx, prob, counts, losses(lg, counts, k, c)


def losses(lg, counts, k, c):
    """The two losses with the counts held fixed (what their gradient differentiates)."""
    E = lg.shape[1]
    n = int(c.sum())
    if n == 0:
        return np.zeros(2)
    p, lse = softmax_rows(lg)
    return np.array([E / (k * n * n) * float((counts * p[c].sum(axis=0)).sum()), float((lse[c] ** 2).sum()) / n])


def backward(logits, idx, prob, counts, dprob=None, dlosses=None, mask=None):
    """dlogits [T, E], and a bound on what its terms sum to in magnitude (for rounding errors)."""
    lg = _rows(logits)
    T, E = lg.shape
    k = idx.shape[1]
    c = counting(lg, mask)
    n = max(int(np.asarray(counts).sum()) // k, 1)
    p, lse = softmax_rows(lg)
    f = E * np.asarray(counts, dtype=np.float64) / (k * n * n)
    d = np.zeros((T, E))
    mag = np.zeros((T, E))
    for t in range(T):
        if dlosses is not None and c[t]:
            gb, gz = float(dlosses[0]), float(dlosses[1])
            jac = np.diag(p[t]) - np.outer(p[t], p[t])
            d[t] += gb * (jac @ f) + gz * (2.0 / n) * lse[t] * p[t]
            mag[t] += abs(gb) * p[t] * (f + p[t] @ f) + abs(gz) * (2.0 / n) * abs(lse[t]) * p[t]
        if dprob is not None:
            w, g = np.asarray(prob[t], dtype=np.float64), np.asarray(dprob[t], dtype=np.float64)
            s = w * (g - w @ g)
            a = w * (np.abs(g) + w @ np.abs(g))
            for j, e in enumerate(idx[t]):
                if 0 <= e < E:
                    d[t, e] += s[j]
                    mag[t, e] += a[j]
    return d, mag

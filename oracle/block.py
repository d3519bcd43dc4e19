"""FP8 with one fp32 scale per block of 128, in numpy -- TEST INFRASTRUCTURE ONLY.

    amax = max |v| of the block;  d = amax / 448, f = 448 / amax  (fp32 divisions, d >= 2^-126,
    f <= 2^126; amax = 0: d = f = 1);  code = E4M3FN(fp32(v f));  value = decode(code) d
"""
from __future__ import annotations

import numpy as np

from . import numerics as nm

B = 128


def block_scale(amax):
    """(f, d) as fp32 arrays of the blocks' amax."""
    a = np.asarray(amax, dtype=np.float32)
    one = np.where(a == 0, np.float32(1), a)
    with np.errstate(over="ignore"):
        f = np.minimum(np.float32(448) / one, np.float32(2.0 ** 126))
    d = np.maximum(one / np.float32(448), np.float32(2.0 ** -126))
    return np.where(a == 0, np.float32(1), f), np.where(a == 0, np.float32(1), d)


def _codes(v32, f):
    return nm.encode_e4m3(nm.round_e4m3((v32 * f).astype(np.float64)))


def quantize_rows(x):
    """x [R, C] (fp32-exact values) -> codes [R, C], scales [C/128, R]."""
    v = np.asarray(x, dtype=np.float32)
    R, C = v.shape
    v = v.reshape(R, C // B, B)
    f, d = block_scale(np.abs(v).max(axis=2))
    return _codes(v, f[:, :, None]).reshape(R, C), np.ascontiguousarray(d.T)


def values_rows(codes, scales):
    R, C = codes.shape
    v = nm.decode_e4m3(codes).reshape(R, C // B, B) * scales.T.astype(np.float64)[:, :, None]
    return v.reshape(R, C)


def padded_starts(offsets):
    off = np.asarray(offsets, dtype=np.int64)
    return np.concatenate([[0], np.cumsum((np.diff(off) + B - 1) // B * B)])


def quantize_tokens(x, offsets):
    """x [R, C] -> codes [C, P], scales [P/128, C]; segments padded with zeros to whole blocks."""
    v = np.asarray(x, dtype=np.float32)
    R, C = v.shape
    off = np.asarray(offsets, dtype=np.int64)
    P = (R + B - 1) // B * B + B * (len(off) - 1)
    pad = np.zeros((P, C), dtype=np.float32)
    st = padded_starts(off)
    for g in range(len(off) - 1):
        pad[st[g]:st[g] + off[g + 1] - off[g]] = v[off[g]:off[g + 1]]
    pad = pad.reshape(P // B, B, C)
    f, d = block_scale(np.abs(pad).max(axis=1))
    return np.ascontiguousarray(_codes(pad, f[:, None, :]).reshape(P, C).T), d


def values_tokens(codes, scales, offsets):
    """[R, C] values of quantize_tokens' output."""
    C, P = codes.shape
    v = (nm.decode_e4m3(codes).reshape(C, P // B, B) * scales.T.astype(np.float64)[:, :, None]).reshape(C, P)
    off, st = np.asarray(offsets, dtype=np.int64), padded_starts(offsets)
    return np.concatenate([v[:, st[g]:st[g] + off[g + 1] - off[g]].T for g in range(len(off) - 1)])


def quantize_matrix(w):
    """w [N, K] -> codes [N, K], scales [ceil(N/128), K/128]; the last rows may be fewer than 128."""
    v = np.asarray(w, dtype=np.float32)
    N, K = v.shape
    nb = -(-N // B)
    pad = np.zeros((nb * B, K), dtype=np.float32)
    pad[:N] = v
    pad = pad.reshape(nb, B, K // B, B)
    f, d = block_scale(np.abs(pad).max(axis=(1, 3)))
    return _codes(pad, f[:, None, :, None]).reshape(nb * B, K)[:N], d


def values_matrix(codes, scales):
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), B, 0)[:N], B, 1)[:, :K]
    return nm.decode_e4m3(codes) * s


def grouped_gemm(a, a_scales, w, w_scales, offsets):
    """(out [R, N], the sums of magnitudes [R, N]); rows outside the offsets are 0."""
    av = values_rows(a, a_scales)
    out = np.zeros((a.shape[0], w.shape[1]))
    mag = np.zeros_like(out)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        wv = values_matrix(w[e], w_scales[e])
        out[lo:hi] = av[lo:hi] @ wv.T
        mag[lo:hi] = np.abs(av[lo:hi]) @ np.abs(wv).T
    return out, mag


def grouped_wgrad(dyt, dyt_scales, xt, xt_scales, offsets):
    """(dw [E, N, K], the sums of magnitudes)."""
    dy, x = values_tokens(dyt, dyt_scales, offsets), values_tokens(xt, xt_scales, offsets)
    E = len(offsets) - 1
    dw = np.zeros((E, dyt.shape[0], xt.shape[0]))
    mag = np.zeros_like(dw)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        dw[e] = dy[lo:hi].T @ x[lo:hi]
        mag[e] = np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])
    return dw, mag

"""Pins of the fp64 router-loss and block-FP8 oracles: gradients against differences, quantization
against its definition, products against scalar loops."""
import numpy as np
import pytest
import torch

from oracle import balance, block
from oracle import numerics as nm


@pytest.mark.parametrize("T,E,k,masked", [(7, 5, 2, False), (9, 6, 3, True), (3, 1, 1, False), (4, 4, 4, True)])
def test_loss_gradient_against_differences(T, E, k, masked):
    g = np.random.default_rng(5)
    lg = g.standard_normal((T, E))
    mask = (np.arange(T) % 3 != 1) if masked else None
    idx, prob, counts, loss = balance.forward(lg, k, mask)
    c = balance.counting(lg, mask)
    dl = np.array([0.7, 0.3])
    got, _ = balance.backward(lg, idx, prob, counts, None, dl, mask)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            diff = (balance.losses(up, counts, k, c) - balance.losses(dn, counts, k, c)) @ dl / (2 * h)
            assert abs(diff - got[t, e]) < 1e-8, (t, e)


def test_weight_gradient_against_differences():
    g = np.random.default_rng(6)
    lg = g.standard_normal((5, 6))
    idx, prob, counts, _ = balance.forward(lg, 3)
    dp = g.standard_normal(prob.shape)
    got, _ = balance.backward(lg, idx, prob, counts, dp)

    def total(l):
        v = np.take_along_axis(l, idx, axis=1)
        w = np.exp(v - v.max(axis=1, keepdims=True))
        return float((w / w.sum(axis=1, keepdims=True) * dp).sum())

    h = 1e-6
    for t in range(5):
        for e in range(6):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((total(up) - total(dn)) / (2 * h) - got[t, e]) < 1e-8


def test_balanced_routing_has_loss_one_and_empty_batches_none():
    lg = np.eye(4) * 3.0                       # each token prefers its own expert, p sums evenly
    _, _, counts, loss = balance.forward(lg, 1)
    assert counts.tolist() == [1, 1, 1, 1] and abs(loss[0] - 1.0) < 1e-12
    assert balance.forward(lg, 1, np.zeros(4))[3].tolist() == [0.0, 0.0]
    dead = np.full((2, 3), -np.inf)
    idx, prob, counts, loss = balance.forward(dead, 2)
    assert idx.tolist() == [[0, 1], [0, 1]] and not prob.any() and not counts.any() and not loss.any()


def test_block_scale_edges():
    tiny = 2.0 ** -126
    f, d = block.block_scale(np.array([0.0, 448.0, 1.0, 1e-45, 3.4e38], dtype=np.float32))
    assert f[0] == 1 and d[0] == 1 and f[1] == 1 and d[1] == 1
    assert f[2] == 448 and d[2] == np.float32(1) / np.float32(448)
    assert f[3] == np.float32(2.0 ** 126) and d[3] == np.float32(tiny)
    assert np.isfinite(f).all() and np.isfinite(d).all() and (f[4] > 0)


@pytest.mark.parametrize("exp", [-140, -60, 0, 100])
def test_block_values_are_within_half_a_step(exp):
    # E4M3 has 3 mantissa bits: half a step is 2^-4 of the value, or of the smallest normal below it;
    # the two fp32 quotients add at most 3 * 2^-24
    g = np.random.default_rng(8)
    x = (g.standard_normal((5, 256)) * 2.0 ** exp).astype(np.float32)
    q, s = block.quantize_rows(x)
    err = np.abs(block.values_rows(q, s) - x)
    d = np.repeat(s.T.astype(np.float64), 128, axis=1)
    assert (err <= np.maximum(np.abs(x.astype(np.float64)), d * 2.0 ** -6) * (2.0 ** -4 + 2.0 ** -22)).all()


def test_layouts_agree_with_scalar_loops():
    g = np.random.default_rng(9)
    off = np.array([0, 3, 3, 140])
    x = torch.from_numpy(g.standard_normal((140, 16))).to(torch.bfloat16).to(torch.float64).numpy()
    q, s = block.quantize_tokens(x, off)
    assert q.shape == (16, 640) and s.shape == (5, 16)
    for col in (0, 7, 15):
        assert s[0, col] == np.float32(np.abs(x[:3, col]).max()) / np.float32(448)
        assert s[1, col] == np.float32(np.abs(x[3:131, col]).max()) / np.float32(448)
        assert s[2, col] == np.float32(np.abs(x[131:, col]).max()) / np.float32(448)
        assert s[3, col] == 1 and not q[col, 128 + 137:].any() and not q[col, 3:128].any()
    w = g.standard_normal((144, 256)).astype(np.float32)
    qm, sm = block.quantize_matrix(w)
    assert sm.shape == (2, 2) and sm[1, 0] == np.float32(np.abs(w[128:, :128]).max()) / np.float32(448)
    qr, sr = block.quantize_rows(g.standard_normal((4, 256)).astype(np.float32))
    out, _ = block.grouped_gemm(qr, sr, qm[None], sm[None], np.array([1, 3]))
    want = sum(nm.decode_e4m3(qr[2, i]) * float(sr[i // 128, 2]) * nm.decode_e4m3(qm[130, i]) * float(sm[1, i // 128])
               for i in range(256))
    assert abs(out[2, 130] - want) < 1e-9 and not out[0].any() and not out[3].any()

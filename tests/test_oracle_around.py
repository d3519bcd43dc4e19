"""The fp64 oracles of grouped routing, the RMS norm and clipping against differences, torch and hand-made cases."""
import numpy as np
import pytest
import torch

from oracle import group_route, norm


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(score, renormalize):
    g = np.random.default_rng(3)
    lg = g.standard_normal((5, 12)) * 1.5
    idx, prob, _ = group_route.forward(lg, 4, g.standard_normal(12) * 0.1, score, 3, 2, 2, renormalize, 2.5)
    dp = g.standard_normal(prob.shape)
    d, mag = group_route.backward(lg, idx, prob, dp, score, renormalize, 2.5)
    h = 1e-6
    for t in range(5):
        for e in range(12):
            up, down = lg.copy(), lg.copy()
            up[t, e] += h
            down[t, e] -= h
            f = [float((group_route.weights(x, idx, score, renormalize, 2.5) * dp).sum()) for x in (up, down)]
            # central differences: h^2 of a third derivative of order 10, and 1e-15 / h
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) <= 1e-8
    assert (np.abs(d) <= mag + 1e-15).all()


def test_groups_by_hand():
    lg = np.log(np.array([[0.1, 0.5, 0.3, 0.3, 0.6, 0.01]]))
    p = np.exp(lg[0]) / np.exp(lg[0]).sum()
    # sums of two: 0.6, 0.6, 0.61 -> groups 2 and 0 (the lower of equal ones); best one: 0.5, 0.3, 0.6
    idx, prob, counts = group_route.forward(lg, 3, None, "softmax", 3, 2, 2, False)
    assert idx[0].tolist() == [4, 1, 0] and np.allclose(prob[0], p[[4, 1, 0]])
    idx, _, _ = group_route.forward(lg, 2, None, "softmax", 3, 1, 1, False)
    assert idx[0].tolist() == [4, 5]
    # the bias counts in the selection alone
    idx, prob, _ = group_route.forward(lg, 1, np.array([5.0, 0, 0, 0, 0, 0]), "softmax", 1, 1, 1, False)
    assert idx[0].tolist() == [0] and np.allclose(prob[0], p[0])
    assert counts.tolist() == [1, 1, 0, 0, 1, 0]


def test_masked_experts_and_rows():
    lg = np.full((3, 4), -np.inf)
    lg[1, 2] = 0.5
    lg[2] = [np.nan, 1.0, np.nan, 3.0]
    idx, prob, _ = group_route.forward(lg, 2)
    assert idx.tolist() == [[0, 1], [2, 0], [0, 2]]
    assert prob[0].tolist() == [0.0, 0.0] and prob[1].tolist() == [1.0, 0.0] and np.isnan(prob[2]).all()


def test_norm_gradient_against_differences_and_autograd():
    g = np.random.default_rng(5)
    s, w, dy, ds = g.standard_normal((3, 7)), 1 + 0.1 * g.standard_normal(7), g.standard_normal((3, 7)), g.standard_normal((3, 7))
    dx, dw, _, _ = norm.backward(dy, s, w, 1e-6, ds)
    h = 1e-6
    for t in range(3):
        for i in range(7):
            f = []
            for d in (h, -h):
                x = s.copy()
                x[t, i] += d
                f.append(float((norm.forward(x, w, 1e-6) * dy).sum() + (x * ds).sum()))
            assert abs((f[0] - f[1]) / (2 * h) - dx[t, i]) <= 1e-7
    a, b = torch.from_numpy(s).requires_grad_(), torch.from_numpy(w).requires_grad_()
    y = a * torch.rsqrt(a.square().mean(1, keepdim=True) + 1e-6) * b
    (y * torch.from_numpy(dy) + a * torch.from_numpy(ds)).sum().backward()
    assert np.allclose(a.grad.numpy(), dx, atol=1e-12) and np.allclose(b.grad.numpy(), dw, atol=1e-12)


def test_clip_as_torch_does():
    g = np.random.default_rng(6)
    grads = [g.standard_normal(n) for n in (5, 1, 300)]
    for m in (0.5, 1e3):
        p = [torch.nn.Parameter(torch.zeros(x.size, dtype=torch.float64)) for x in grads]
        for q, x in zip(p, grads):
            q.grad = torch.from_numpy(x.copy())
        total = torch.nn.utils.clip_grad_norm_(p, m)
        n, out = norm.clip(grads, m)
        assert abs(float(total) - n) <= 1e-12 * n
        for q, x in zip(p, out):
            assert np.allclose(q.grad.numpy(), x, rtol=1e-12, atol=0)

"""GPU parity of grouped routing (moe_route_grouped and its gradient) against the fp64 oracle.

Ids and counts are compared exactly: the order is that of 64-bit scores, whose distances in these inputs are far above
what two 64-bit exponentials differ by.  Tolerances, u = 2^-24: the exponential is the hardware's exp2 of x log2 e,
off by (|x| + 2) u, with |x| <= 12 here (a difference of logits, or a logit whose score is not next to 1), its sum
with 1 and the reciprocal 4 u: a score is within 18 u of itself; a sum of scores of one sign within 18 u + 16 u;
quotient and scale 4 u: a weight within 56 u of itself, 80 u allowed.  A gradient's terms are products of such
factors with sums of at most 16 terms: within 96 u of the sum of their magnitudes, and half an output step.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, log, need_gpu
from oracle import group_route

U = 2.0 ** -24
TINY = 2.0 ** -126      # results below the smallest normal number may be flushed


def _logits(T, E, kind, dtype, seed=3):
    g = np.random.default_rng(seed + 7 * T + E)
    lg = g.standard_normal((T, E)) * 1.5
    if kind == "ties":
        lg = np.round(lg)
    elif kind == "zeros":
        lg = np.where(g.random((T, E)) < 0.5, 0.0, -0.0)
    elif kind == "masked-experts":
        lg[:, :: 3] = -np.inf
    elif kind == "lowest":
        lg[:, 1:: 2] = float(torch.finfo(dtype).min)
    elif kind == "dead-rows":
        lg[:: 2] = -np.inf
        lg[1:: 4, 2:] = -np.inf
    elif kind == "tiny-scores":
        lg = lg - 95.0
    elif kind == "saturated":
        lg = lg + 30.0
    return torch.from_numpy(lg.astype(np.float32)).to(dtype)


F, B = torch.float32, torch.bfloat16
CASES = [
    # T, E, k, G, kg, best, score, bias, renorm, scale, kind, dtype, masked
    (1, 1, 1, 1, 1, 1, "sigmoid", False, True, 1.0, "normal", F, False),
    (1, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5, "normal", F, False),
    (3, 2, 2, 2, 2, 1, "softmax", True, False, 1.0, "normal", F, True),
    (5, 7, 7, 1, 1, 1, "sigmoid", True, True, 1.0, "ties", B, False),
    (257, 8, 2, 4, 2, 2, "sigmoid", True, True, 1.0, "normal", B, True),
    (129, 9, 3, 3, 1, 2, "softmax", False, True, 1.0, "ties", F, False),
    (513, 16, 1, 16, 3, 1, "sigmoid", True, False, 1.0, "normal", F, True),
    (400, 32, 16, 16, 8, 2, "softmax", True, True, 16.0, "normal", F, True),
    (1000, 18, 5, 6, 4, 2, "sigmoid", False, True, 1.0, "masked-experts", F, False),
    (300, 48, 6, 3, 2, 1, "softmax", True, False, 1.0, "masked-experts", B, True),
    (700, 30, 16, 5, 3, 2, "sigmoid", False, True, 1.0, "zeros", B, False),
    (400, 33, 9, 11, 5, 2, "softmax", False, False, 2.5, "zeros", F, True),
    (900, 64, 8, 4, 2, 2, "sigmoid", True, True, 2.5, "normal", B, True),
    (640, 64, 8, 8, 3, 1, "sigmoid", False, True, 1.0, "ties", B, True),
    (500, 100, 7, 10, 3, 2, "sigmoid", True, False, 1.0, "normal", F, True),
    (300, 129, 12, 3, 2, 2, "softmax", True, True, 1.0, "normal", F, False),
    (333, 160, 6, 8, 3, 1, "softmax", False, False, 16.0, "normal", B, False),
    (2000, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5, "normal", F, True),
    (333, 256, 16, 16, 2, 2, "sigmoid", False, True, 1.0, "normal", B, False),
    (333, 256, 16, 1, 1, 1, "sigmoid", False, True, 1.0, "normal", F, False),
    (250, 251, 5, 1, 1, 1, "softmax", True, True, 1.0, "normal", B, False),
    (300, 200, 4, 2, 1, 2, "sigmoid", True, True, 1.0, "lowest", F, False),
    (300, 200, 4, 2, 1, 2, "softmax", False, True, 1.0, "lowest", F, False),
    (200, 6, 4, 3, 2, 2, "sigmoid", False, True, 1.0, "dead-rows", F, True),
    (200, 6, 4, 3, 2, 1, "softmax", True, False, 1.0, "dead-rows", B, True),
    (200, 40, 4, 4, 2, 2, "sigmoid", False, True, 1.0, "tiny-scores", F, False),
    (200, 40, 4, 4, 2, 2, "sigmoid", True, False, 1.0, "tiny-scores", F, False),
    (200, 40, 4, 4, 2, 1, "sigmoid", True, True, 1.0, "saturated", F, False),
    (9001, 24, 4, 6, 3, 2, "sigmoid", True, True, 1.0, "normal", F, True),
    (20993, 12, 4, 1, 1, 1, "softmax", True, True, 1.0, "normal", B, True),
]
IDS = [f"T{c[0]}-E{c[1]}-k{c[2]}-G{c[3]}.{c[4]}.{c[5]}-{c[6]}{'-bias' if c[7] else ''}{'' if c[8] else '-plain'}-{c[10]}-"
       f"{'f32' if c[11] == F else 'bf16'}{'-mask' if c[12] else ''}" for c in CASES]


def _bias(E, kind, seed=5):
    return torch.from_numpy((np.random.default_rng(seed + E).standard_normal(E) * 0.1).astype(np.float32))


def _mask(T, masked):
    return torch.from_numpy(np.random.default_rng(T).random(T) < 0.8) if masked else None


def _gpu(t):
    return None if t is None else t.cuda()


def _close(got, want, tol):
    assert ((np.abs(got - want) <= tol) | ((got == want) | (np.isnan(got) & np.isnan(want)))).all(), \
        float(np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300)))


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_gradient(case):
    m = need_gpu()
    T, E, k, G, kg, best, score, bias, renorm, scale, kind, dtype, masked = case
    lg, mask, b = _logits(T, E, kind, dtype), _mask(T, masked), _bias(E, kind) if bias else None
    kw = dict(score=score, groups=G, topk_groups=kg, group_best=best, renormalize=renorm, scale=scale)
    idx, prob, counts = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), token_mask=_gpu(mask), count=True, **kw)
    i2, p2, none = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), **kw)
    torch.cuda.synchronize()
    assert none is None and torch.equal(idx, i2) and torch.equal(prob, p2)
    ri, rp, rc = group_route.forward(lg, k, b, mask=None if mask is None else mask.numpy(), **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    got = prob.cpu().double().numpy()
    log(f"weights off by at most {np.max(np.abs(got - rp) / np.maximum(rp, TINY)) / U:.1f} u")
    _close(got, rp, 80 * U * rp + TINY * scale)
    # the gradient, from the kernel's own ids and weights
    dp = torch.from_numpy(np.random.default_rng(1).standard_normal((T, k)).astype(np.float32))
    out = m.moe_route_grouped_bwd(lg.cuda(), idx, prob, dp.cuda(), score=score, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    assert out.dtype == dtype
    want, mag = group_route.backward(lg, ri, prob.cpu().numpy(), dp.numpy(), score, renorm, scale)
    _close(out.cpu().double().numpy(), want,
           96 * U * mag + np.abs(want) * float(torch.finfo(dtype).eps) / 2 + TINY * 16 * scale)


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G", [(40, 1), (256, 8), (96, 3)])
def test_nearly_equal_scores_take_their_64_bit_order(score, E, G):
    """Biases that make every score + bias equal to within fp32's rounding: 32-bit values would tie or swap."""
    m = need_gpu()
    g = np.random.default_rng(E + G)
    T, k = 37, min(8, E // G)
    base = (g.standard_normal(E) * 1.5).astype(np.float32)
    lg = np.repeat(base[None], T, 0)
    lg[1::3] = (g.standard_normal((len(lg[1::3]), E)) * 1.5).astype(np.float32)       # ordinary rows between
    s = group_route.scores(base[None].astype(np.float64), score)[0]
    b = (0.9 - s).astype(np.float32)
    c = s + b.astype(np.float64)
    assert 0 < np.diff(np.sort(c)).min() and np.ptp(c) < 1.3e-7
    kw = dict(score=score, groups=G, topk_groups=max(1, G // 2), group_best=2 if G > 1 else 1)
    idx, prob, _ = m.moe_route_grouped(torch.from_numpy(lg).cuda(), k, bias=torch.from_numpy(b).cuda(), **kw)
    torch.cuda.synchronize()
    ri, rp, _ = group_route.forward(lg, k, b, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    _close(prob.cpu().double().numpy(), rp, 80 * U * rp)


@gpu
@pytest.mark.parametrize("dtype", [F, B], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,k,G,kg,best", [(7, 2, 1, 1, 1), (32, 4, 8, 3, 2), (256, 8, 8, 4, 2), (60, 16, 4, 2, 1)])
def test_nan_infinity_and_large_biases(dtype, E, k, G, kg, best):
    m = need_gpu()
    lg = _logits(40, E, "normal", dtype)
    nan, inf = float("nan"), float("inf")
    lg[1, E - 1], lg[2, 3], lg[3, E // 2], lg[4, 0], lg[5, 1] = nan, inf, -inf, -nan, inf
    lg[5, E - 2] = nan
    lg[6] = nan
    for score in ("sigmoid", "softmax"):
        for b in (None, torch.zeros(E), torch.linspace(-300, 300, E), torch.full((E,), -inf), torch.full((E,), 1e30)):
            if b is not None and E > 30 and abs(float(b[0])) < 1e3:
                b[5], b[9], b[11] = inf, -inf, nan
            kw = dict(score=score, groups=G, topk_groups=kg, group_best=best)
            idx, prob, _ = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), **kw)
            torch.cuda.synchronize()
            ri, rp, _ = group_route.forward(lg, k, b, **kw)
            np.testing.assert_array_equal(idx.cpu().numpy(), ri)
            _close(prob.cpu().double().numpy(), rp, 80 * U * rp + TINY)


@gpu
@pytest.mark.parametrize("dtype", [F, B], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,G,kg,k,best", [(256, 8, 4, 8, 2), (256, 8, 3, 8, 1), (256, 2, 1, 16, 2), (250, 2, 1, 3, 1),
                                           (240, 16, 8, 6, 2), (255, 5, 2, 16, 2), (128, 16, 1, 5, 1), (99, 3, 1, 8, 2),
                                           (64, 4, 2, 8, 2), (256, 4, 1, 2, 2), (252, 7, 3, 12, 1)])
def test_few_groups_of_many_tokens(E, G, kg, k, best, dtype):
    """Half of the groups or fewer, with rows that hold ties, NaN and infinities between ordinary ones."""
    m = need_gpu()
    T = 5003
    lg = _logits(T, E, "normal", dtype)
    lg[1::5] = torch.round(lg[1::5].float()).to(dtype)
    lg[2::7, ::3] = -float("inf")
    lg[3::11] = -float("inf")
    lg[4::13, E - 1] = float("nan")
    lg[5::17, E // 2] = float("inf")
    for score in ("sigmoid", "softmax"):
        for b in (None, _bias(E, "normal")):
            kw = dict(score=score, groups=G, topk_groups=kg, group_best=best)
            idx, prob, counts = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), count=True, **kw)
            torch.cuda.synchronize()
            ri, rp, rc = group_route.forward(lg, k, b, **kw)
            np.testing.assert_array_equal(idx.cpu().numpy(), ri)
            np.testing.assert_array_equal(counts.cpu().numpy(), rc)
            _close(prob.cpu().double().numpy(), rp, 80 * U * rp + TINY)


@gpu
@pytest.mark.parametrize("dtype", [F, B], ids=["f32", "bf16"])
def test_equal_scores_go_by_their_ids(dtype):
    """Whole rows of equal logits, and biases that repeat, as routers begin: through the fp32 order and the 64-bit one."""
    m = need_gpu()
    g = np.random.default_rng(9)
    for T, E, k, G, kg, best in ((50, 64, 8, 8, 3, 2), (5000, 64, 6, 1, 1, 1), (4500, 256, 8, 8, 4, 2), (4200, 48, 4, 3, 2, 1)):
        lg = np.zeros((T, E))
        lg[1::3] = np.round(g.standard_normal((len(lg[1::3]), E)) * 2) / 2
        lg[2::3] = g.standard_normal((len(lg[2::3]), E)) * 1.5
        b = torch.from_numpy(np.round(g.standard_normal(E) * 3).astype(np.float32) * np.float32(0.001))
        t = torch.from_numpy(lg.astype(np.float32)).to(dtype)
        for bias in (None, b, torch.zeros(E)):
            for score in ("sigmoid", "softmax"):
                kw = dict(score=score, groups=G, topk_groups=kg, group_best=best)
                idx, prob, counts = m.moe_route_grouped(t.cuda(), k, bias=_gpu(bias), count=True, **kw)
                torch.cuda.synchronize()
                rows = np.r_[0:60, T - 60:T] if T > 120 else np.arange(T)
                ri, rp, _ = group_route.forward(t[rows], k, bias, **kw)
                np.testing.assert_array_equal(idx.cpu().numpy()[rows], ri)
                _close(prob.cpu().double().numpy()[rows], rp, 80 * U * rp)
                assert torch.equal(counts.long(), torch.bincount(idx.reshape(-1).long(), minlength=E))


@gpu
def test_biases_that_differ_by_less_than_their_distance_from_the_lowest_shows():
    """1 + 2^-23 and 1 are the same over -3 in fp32: with equal logits the larger bias still goes first."""
    m = need_gpu()
    b = torch.ones(32)
    b[20] += 2.0 ** -23
    b[3] = -3.0
    for T in (3, 5000):
        lg = torch.zeros((T, 32))
        idx, _, _ = m.moe_route_grouped(lg.cuda(), 3, bias=b.cuda())
        torch.cuda.synchronize()
        assert (idx.cpu() == torch.tensor([20, 0, 1], dtype=torch.int32)).all()


@gpu
def test_softmax_without_groups_is_the_plain_router():
    m = need_gpu()
    for T, E, k, dtype in ((5000, 8, 2, F), (3001, 64, 8, B), (777, 256, 16, F)):
        lg = _logits(T, E, "ties", dtype).cuda()
        idx, prob, counts = m.moe_route_grouped(lg, k, score="softmax", count=True)
        i2, p2, c2, _ = m.moe_route_balance(lg, k)
        torch.cuda.synchronize()
        assert torch.equal(idx, i2) and torch.equal(counts, c2)
        assert float((prob - p2).abs().max()) <= 120 * U


@gpu
def test_repeated_and_foreign_ids_in_the_gradient():
    m = need_gpu()
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            for dtype in (F, B):
                lg = _logits(23, 9, "normal", dtype)
                g = np.random.default_rng(2)
                idx = torch.from_numpy(g.integers(0, 9, (23, 5)).astype(np.int32))
                idx[2::3, 0], idx[2::3, 3], idx[::4, 1] = -1, 9, 2 ** 31 - 1
                idx[7] = 4
                prob = torch.from_numpy(g.random((23, 5)).astype(np.float32))
                dp = torch.from_numpy(g.standard_normal((23, 5)).astype(np.float32))
                out = m.moe_route_grouped_bwd(lg.cuda(), idx.cuda(), prob.cuda(), dp.cuda(), score=score, renormalize=renorm,
                                              scale=1.5)
                again = m.moe_route_grouped_bwd(lg.cuda(), idx.cuda(), prob.cuda(), dp.cuda(), score=score,
                                                renormalize=renorm, scale=1.5)
                torch.cuda.synchronize()
                assert torch.equal(out, again)
                want, mag = group_route.backward(lg, idx.numpy(), prob.numpy(), dp.numpy(), score, renorm, 1.5)
                _close(out.cpu().double().numpy(), want, 96 * U * mag + np.abs(want) * float(torch.finfo(dtype).eps) / 2 + TINY)


@gpu
def test_one_renormalised_slot_has_no_gradient():
    """Its weight is the scale whatever the logits are: zeros, not what rounding leaves of a difference."""
    m = need_gpu()
    for score in ("sigmoid", "softmax"):
        for scale in (1.0, 2.5, 0.1, 16.0):
            for dtype in (F, B):
                lg = _logits(333, 21, "normal", dtype).cuda()
                idx, prob, _ = m.moe_route_grouped(lg, 1, score=score, scale=scale)
                dp = torch.from_numpy(np.random.default_rng(3).standard_normal((333, 1)).astype(np.float32)).cuda()
                out = m.moe_route_grouped_bwd(lg, idx, prob, dp, score=score, scale=scale)
                torch.cuda.synchronize()
                assert not out.any()


@gpu
def test_many_tokens_and_unaligned_logits():
    """More tokens than the kernels hold at once, and logits that begin anywhere."""
    m = need_gpu()
    for T, E, dtype, shift in ((70001, 20, F, 1), (40003, 33, B, 3), (3, 256, B, 1)):
        flat = torch.empty(T * E + 8, dtype=dtype, device="cuda")
        lg = _logits(T, E, "normal", dtype)
        view = flat[shift:shift + T * E].view(T, E)
        view.copy_(lg)
        b = _bias(E, "normal")
        kw = dict(score="sigmoid", groups=1 if E == 33 else 4, topk_groups=1 if E == 33 else 2)
        idx, prob, counts = m.moe_route_grouped(view, 4, bias=b.cuda(), count=True, **kw)
        i2, p2, c2 = m.moe_route_grouped(lg.cuda(), 4, bias=b.cuda(), count=True, **kw)
        out = m.moe_route_grouped_bwd(view, idx, prob, prob)
        o2 = m.moe_route_grouped_bwd(lg.cuda(), idx, prob, prob)
        torch.cuda.synchronize()
        assert torch.equal(idx, i2) and torch.equal(prob, p2) and torch.equal(counts, c2) and torch.equal(out, o2)
        ri, rp, rc = group_route.forward(lg[-2000:], 4, b, group_best=2, **kw)
        np.testing.assert_array_equal(idx[-2000:].cpu().numpy(), ri)
        assert int(counts.sum()) == 4 * T


@gpu
def test_deterministic_on_two_streams_and_in_two_graphs():
    m = need_gpu()
    lg, lg2 = _logits(9000, 64, "normal", F).cuda(), _logits(5000, 32, "ties", B).cuda()
    b, b2 = _bias(64, "normal").cuda(), _bias(32, "normal").cuda()

    def step(x, bias, k):
        idx, prob, counts = m.moe_route_grouped(x, k, bias=bias, groups=4, topk_groups=2, count=True)
        return idx, prob, counts, m.moe_route_grouped_bwd(x, idx, prob, prob)

    want, want2 = step(lg, b, 8), step(lg2, b2, 4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        a = step(lg, b, 8)
    with torch.cuda.stream(s2):
        c = step(lg2, b2, 4)
    torch.cuda.synchronize()
    for got, ref in ((a, want), (c, want2)):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = step(lg, b, 8)
    with torch.cuda.graph(g2):
        c = step(lg2, b2, 4)
    for _ in range(3):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        step(lg2, b2, 8)
        torch.cuda.synchronize()
        for got, ref in ((a, want), (c, want2)):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))


@gpu
def test_refusals_on_the_gpu():
    m = need_gpu()
    lg = torch.zeros((6, 8), device="cuda")
    idx, prob, _ = m.moe_route_grouped(lg, 2)
    for kw in (dict(k=9), dict(k=0), dict(groups=3), dict(groups=0), dict(groups=4, topk_groups=1, k=3),
               dict(groups=8, group_best=2), dict(scale=0.0), dict(topk_groups=2)):
        with pytest.raises(m.MoeError):
            m.moe_route_grouped(lg, **{"k": 2, **kw})
    with pytest.raises(ValueError):
        m.moe_route_grouped(lg, 2, score="tanh")
    with pytest.raises(ValueError):
        m.moe_route_grouped(lg, 2, token_mask=torch.ones(6, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        m.moe_route_grouped(lg, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(TypeError):
        m.moe_route_grouped(lg, 2, bias=torch.zeros(8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m.moe_route_grouped(lg, 2, bias=torch.zeros(8))
    with pytest.raises(TypeError):
        m.moe_route_grouped(lg.half(), 2)
    with pytest.raises(ValueError):
        m.moe_route_grouped(lg.t(), 2)
    with pytest.raises(ValueError):
        m.moe_route_grouped_bwd(lg, idx, prob[:5], prob)
    with pytest.raises(TypeError):
        m.moe_route_grouped_bwd(lg, idx.long(), prob, prob)
    with pytest.raises(m.MoeError):
        m.moe_route_grouped_bwd(lg, idx, prob, prob, scale=-1.0)
    with pytest.raises(m.MoeError):
        m.moe_route_grouped(torch.zeros((0, 8), device="cuda"), 2)


@gpu
@pytest.mark.parametrize("dtype", [F, B], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 5003])
@pytest.mark.parametrize("E,k,G,kg,best", [(16, 4, 1, 1, 1), (64, 8, 8, 4, 2), (256, 8, 1, 1, 1), (256, 6, 8, 5, 1)])
def test_rows_of_very_low_logits(E, k, G, kg, best, T, dtype):
    """Whole rows whose sigmoids are 0 in 64 bits (below -709.78, a padding token's lowest value among them) have no weight
    and no gradient, whichever way a token takes; of the lowest that are not the ratios stay.  Softmax scores likewise,
    where a bias selects what lies far below the row's largest."""
    m = need_gpu()
    g = np.random.default_rng(E)
    lg = g.standard_normal((T, E)) * 1.5
    low = np.arange(T) % 10
    lg[low == 1] = float(torch.finfo(dtype).min)
    lg[low == 2] = -1000.0
    lg[low == 3] = -1000.0 - 64 * np.round(g.random(((low == 3).sum(), E)) * 60)
    lg[low == 4] = -712.0 + 8 * np.round(g.random(((low == 4).sum(), E)))          # 0 or not, experts apart
    lg[low == 5] -= 500.0
    lg[low == 6] = -5000.0                                                         # softmax: all alike
    lg[low == 7, : E // 2] -= 1000.0                                               # half of them far below
    lg[low == 8, : E // 2] -= 600.0
    t = torch.from_numpy(lg.astype(np.float32)).to(dtype)
    rows = np.r_[0:80, T - 40:T] if T > 120 else np.arange(T)
    first = torch.where(torch.arange(E) < E // 2, 3.0, 0.0)                        # selects the lower half
    for score in ("sigmoid", "softmax"):
        for b in (None, _bias(E, "normal"), torch.zeros(E), _bias(E, "normal") + first):
            for renorm in (True, False):
                kw = dict(score=score, groups=G, topk_groups=kg, group_best=best, renormalize=renorm, scale=2.5)
                idx, prob, counts = m.moe_route_grouped(t.cuda(), k, bias=_gpu(b), count=True, **kw)
                dp = torch.from_numpy(np.random.default_rng(1).standard_normal((T, k)).astype(np.float32))
                out = m.moe_route_grouped_bwd(t.cuda(), idx, prob, dp.cuda(), score=score, renormalize=renorm, scale=2.5)
                torch.cuda.synchronize()
                ri, rp, _ = group_route.forward(t[rows], k, b, **kw)
                log(f"{score} bias {b is not None} renorm {renorm}")
                np.testing.assert_array_equal(idx.cpu().numpy()[rows], ri)
                _close(prob.cpu().double().numpy()[rows], rp, 80 * U * rp + TINY * 2.5)
                assert torch.equal(counts.long(), torch.bincount(idx.reshape(-1).long(), minlength=E))
                if score == "sigmoid":
                    none = torch.from_numpy((low >= 1) & (low <= 3)).cuda()
                    assert not prob[none].any() and not out[none].any()


@gpu
@pytest.mark.parametrize("k", [2, 3, 8, 13])
@pytest.mark.parametrize("E,G,kg,best", [
    (16, 1, 1, 1), (32, 1, 1, 1), (60, 1, 1, 1), (65, 1, 1, 1), (128, 1, 1, 1), (129, 1, 1, 1), (256, 1, 1, 1),   # no groups
    (16, 16, 14, 1), (32, 16, 9, 2), (60, 15, 8, 2), (80, 16, 9, 1), (128, 4, 3, 2), (240, 8, 5, 2),             # over half of them
    (256, 2, 2, 2), (255, 3, 2, 2), (255, 5, 3, 1), (252, 9, 5, 2),
    (64, 4, 2, 2), (128, 16, 8, 1), (256, 16, 8, 2), (255, 3, 1, 2)])                                             # half or fewer
def test_many_tokens_of_each_width(E, G, kg, best, k):
    """Each count of experts a lane (1 to 32), with and without the halving of groups, by each length of list, in one launch
    and at more tokens than one does to the end; rows that hold ties, NaN and infinities between ordinary ones.  And the
    gradient at those widths."""
    m = need_gpu()
    for T, dtype in ((97, F), (97, B), (4099, F), (4099, B)):
        rows = np.arange(T) if T < 1000 else np.r_[0:150, 2000:2050, T - 60:T]
        mask = torch.from_numpy(np.random.default_rng(E).random(T) < 0.7)
        dp = torch.from_numpy(np.random.default_rng(k).standard_normal((T, k)).astype(np.float32))
        lg = _logits(T, E, "normal", dtype)
        lg[1::5] = torch.round(lg[1::5].float()).to(dtype)
        lg[2::7, ::3] = -float("inf")
        lg[3::11] = -float("inf")
        lg[4::13, E - 1] = float("nan")
        lg[5::17, E // 2] = float("inf")
        for score, b, renorm in (("sigmoid", None, True), ("sigmoid", _bias(E, "normal"), True),
                                 ("softmax", None, False), ("softmax", _bias(E, "normal") * 0.1, True)):
            kw = dict(score=score, groups=G, topk_groups=kg, group_best=best, renormalize=renorm)
            idx, prob, counts = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), count=True, token_mask=mask.cuda(), **kw)
            i2, p2, _ = m.moe_route_grouped(lg.cuda(), k, bias=_gpu(b), **kw)
            out = m.moe_route_grouped_bwd(lg.cuda(), idx, prob, dp.cuda(), score=score, renormalize=renorm)
            torch.cuda.synchronize()
            assert torch.equal(idx, i2) and torch.equal(prob.nan_to_num(7.0), p2.nan_to_num(7.0))
            log(f"{T} x {E} {score} bias {b is not None}")
            ri, rp, _ = group_route.forward(lg[rows], k, b, **kw)
            np.testing.assert_array_equal(idx.cpu().numpy()[rows], ri)
            _close(prob.cpu().double().numpy()[rows], rp, 80 * U * rp + TINY)
            live = idx.cpu()[mask].reshape(-1).long()
            assert torch.equal(counts.cpu().long(), torch.bincount(live, minlength=E))
            want, mag = group_route.backward(lg[rows], ri, prob.cpu().numpy()[rows], dp.numpy()[rows], score, renorm)
            _close(out.cpu().double().numpy()[rows], want,
                   96 * U * mag + np.abs(want) * float(torch.finfo(dtype).eps) / 2 + TINY * 16)

"""GPU parity of the training router (moe_route_balance and its gradient) against the fp64 oracle.

Ids and counts are compared bit-exactly.  Tolerances, with u = 2^-24 the fp32 half step:
  * exp is the hardware exp2 of x log2 e, off by up to (|x| + 2) u relative; logits here differ by at
    most 20, so p and w are within 24 u + the sum's 16 u < 40 u relative: PROB 40 u absolute (p <= 1),
    and 80 u relative for the losses (lse^2 doubles its error; the sums over tokens are 64-bit past a
    block of fp32 sums of same-signed terms);
  * a gradient is a sum of terms each within 48 u of itself (p, the weights, lse and the products):
    48 u times the sum of their magnitudes, and half an output step.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, log, need_gpu
from oracle import balance

U = 2.0 ** -24


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
    t = torch.from_numpy(lg.astype(np.float32)).to(dtype)
    return t


CASES = [
    # T, E, k, kind, dtype, masked
    (1, 1, 1, "normal", torch.float32, False),
    (1, 8, 2, "normal", torch.bfloat16, False),
    (3, 2, 2, "normal", torch.float32, True),
    (256, 4, 2, "normal", torch.float32, False),
    (257, 8, 8, "ties", torch.bfloat16, True),
    (129, 9, 3, "ties", torch.float32, False),
    (513, 16, 16, "normal", torch.float32, True),
    (1000, 17, 5, "masked-experts", torch.float32, False),
    (700, 31, 16, "zeros", torch.bfloat16, False),
    (400, 33, 9, "zeros", torch.float32, True),
    (900, 64, 8, "normal", torch.bfloat16, True),
    (640, 64, 8, "masked-experts", torch.bfloat16, True),
    (500, 100, 7, "ties", torch.float32, True),
    (300, 129, 12, "normal", torch.float32, False),
    (2000, 256, 8, "normal", torch.float32, True),
    (333, 256, 16, "ties", torch.bfloat16, False),
    (300, 200, 1, "lowest", torch.float32, False),
    (200, 6, 4, "dead-rows", torch.float32, True),
    (40000, 12, 4, "normal", torch.float32, True),
]
IDS = [f"T{c[0]}-E{c[1]}-k{c[2]}-{c[3]}-{'f32' if c[4] == torch.float32 else 'bf16'}{'-mask' if c[5] else ''}"
       for c in CASES]


def _mask(T, masked):
    return torch.from_numpy(np.random.default_rng(T).random(T) < 0.8) if masked else None


def _gpu(t):
    return None if t is None else t.cuda()


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_gradient(case):
    m = need_gpu()
    T, E, k, kind, dtype, masked = case
    lg, mask = _logits(T, E, kind, dtype), _mask(T, masked)
    idx, prob, counts, losses = m.moe_route_balance(lg.cuda(), k, token_mask=_gpu(mask))
    torch.cuda.synchronize()
    ri, rp, rc, rl = balance.forward(lg, k, None if mask is None else mask.numpy())
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    assert np.abs(prob.cpu().double().numpy() - rp).max() <= 40 * U
    got = losses.cpu().double().numpy()
    log(f"losses {got} oracle {rl}")
    for a, b in zip(got, rl):
        if b > float(torch.finfo(torch.float32).max):
            assert np.isinf(a)              # lse^2 of rows at the type's lowest value passes fp32
        else:
            assert abs(a - b) <= 80 * U * abs(b) + 1e-30
    # the gradient, from the kernel's own ids and weights
    g = np.random.default_rng(1)
    dprob = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32))
    dl = torch.tensor([0.8, 0.05])
    for dp, d in ((dprob, dl), (dprob, None), (None, dl), (None, None)):
        out = m.moe_route_balance_bwd(lg.cuda(), idx, prob, counts, _gpu(dp), _gpu(d), token_mask=_gpu(mask))
        torch.cuda.synchronize()
        assert out.dtype == dtype
        want, mag = balance.backward(lg, ri, prob.cpu().numpy(), rc, None if dp is None else dp.numpy(),
                                     None if d is None else d.numpy(), None if mask is None else mask.numpy())
        err = np.abs(out.cpu().double().numpy() - want)
        tol = 48 * U * mag + np.abs(want) * float(torch.finfo(dtype).eps) / 2 + 1e-37
        assert (err <= tol).all(), float((err / tol).max())


@gpu
def test_routing_equals_route_topk():
    m = need_gpu()
    for T, E, k, dtype in ((5000, 8, 2, torch.float32), (3001, 64, 8, torch.bfloat16), (777, 256, 16, torch.float32)):
        lg = _logits(T, E, "ties", dtype).cuda()
        idx, prob, counts, _ = m.moe_route_balance(lg, k)
        i2, p2 = m.moe_route_topk(lg, k)
        perm = m.moe_permute(None, idx, prob, E)
        torch.cuda.synchronize()
        assert torch.equal(idx, i2) and torch.equal(counts, perm["split_sizes"])
        assert float((prob - p2).abs().max()) <= 40 * U


@gpu
def test_all_masked_and_nan_rows():
    m = need_gpu()
    lg = _logits(70, 10, "normal", torch.float32).cuda()
    none = torch.zeros(70, dtype=torch.uint8, device="cuda")
    idx, prob, counts, losses = m.moe_route_balance(lg, 3, token_mask=none)
    d = m.moe_route_balance_bwd(lg, idx, prob, counts, None, torch.ones(2, device="cuda"), token_mask=none)
    assert not counts.any() and losses.tolist() == [0.0, 0.0] and not d.any()
    bad = lg.clone()
    bad[4, 7] = float("nan")
    bad[9, 2] = float("inf")
    idx, prob, counts, losses = m.moe_route_balance(bad, 3)
    torch.cuda.synchronize()
    assert idx[4, 0].item() == 7 and idx[9, 0].item() == 2
    assert int(idx.min()) >= 0 and int(idx.max()) < 10 and torch.isnan(losses).all()
    ok = torch.arange(70, device="cuda")
    ok = (ok != 4) & (ok != 9)
    assert torch.isfinite(prob[ok]).all() and torch.isnan(prob[~ok]).all()


@gpu
def test_repeated_and_foreign_ids_in_the_gradient():
    """topk_idx is the caller's array: an id twice gets both parts, one outside [0, E) none."""
    m = need_gpu()
    lg = _logits(20, 5, "normal", torch.float32)
    idx = torch.zeros((20, 2), dtype=torch.int32)
    idx[1::3] = 3
    idx[2::3, 0] = -1
    idx[2::3, 1] = 5
    g = np.random.default_rng(2)
    prob = torch.from_numpy(g.random((20, 2)).astype(np.float32))
    dp = torch.from_numpy(g.standard_normal((20, 2)).astype(np.float32))
    counts = torch.zeros(5, dtype=torch.int32)
    out = m.moe_route_balance_bwd(lg.cuda(), idx.cuda(), prob.cuda(), counts.cuda(), dp.cuda())
    want, mag = balance.backward(lg, idx.numpy(), prob.numpy(), counts.numpy(), dp.numpy())
    assert (np.abs(out.cpu().double().numpy() - want) <= 48 * U * mag + np.abs(want) * U).all()


@gpu
def test_deterministic_on_two_streams_and_in_two_graphs():
    m = need_gpu()
    lg = _logits(9000, 64, "normal", torch.float32).cuda()
    lg2 = _logits(5000, 32, "ties", torch.float32).cuda()
    dl = torch.tensor([0.3, 0.2], device="cuda")

    def step(x, k):
        idx, prob, counts, losses = m.moe_route_balance(x, k)
        return idx, prob, counts, losses, m.moe_route_balance_bwd(x, idx, prob, counts, prob, dl)

    want, want2 = step(lg, 8), step(lg2, 4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        a = step(lg, 8)
    with torch.cuda.stream(s2):
        b = step(lg2, 4)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c = step(lg, 8)
    with torch.cuda.graph(g2):
        d = step(lg2, 4)
    for got, ref in ((a, want), (b, want2)):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    for _ in range(3):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        step(lg2, 8)
        torch.cuda.synchronize()
        for got, ref in ((c, want), (d, want2)):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))


@gpu
def test_refusals_on_the_gpu():
    m = need_gpu()
    lg = torch.zeros((6, 4), device="cuda")
    idx, prob, counts, _ = m.moe_route_balance(lg, 2)
    with pytest.raises(m.MoeError):
        m.moe_route_balance(lg, 5)
    with pytest.raises(TypeError):
        m.moe_route_balance(lg.to(torch.float16), 2)
    with pytest.raises(ValueError):
        m.moe_route_balance(lg.t(), 2)
    with pytest.raises(ValueError):
        m.moe_route_balance(lg, 2, token_mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError):
        m.moe_route_balance(lg, 2, token_mask=torch.ones(6, device="cuda"))
    with pytest.raises(ValueError):
        m.moe_route_balance_bwd(lg, idx, prob[:5], counts)
    with pytest.raises(TypeError):
        m.moe_route_balance_bwd(lg, idx.long(), prob, counts)
    with pytest.raises(ValueError):
        m.moe_route_balance_bwd(lg, idx, prob, counts, dlosses=torch.ones(1, device="cuda"))


# bit patterns of NaN: quiet with either sign, and all ones, what a host's conversion to bf16 writes
NANS = {torch.bfloat16: [0x7FC0, -0x0040, -0x0001, 0x7F81], torch.float32: [0x7FC00000, -0x00400000, -0x00000001, 0x7FC00001]}


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,k", [(7, 2), (10, 3), (30, 4), (64, 8), (256, 8)])
def test_a_nan_of_either_sign_is_selected_first(E, k, dtype):
    """Ahead of everything finite, also at an expert that would be chosen last; the lower id first among
    several, whatever their bits.  The token's weights and both losses are NaN, other tokens as they were."""
    m = need_gpu()
    T = 40
    lg = _logits(T, E, "normal", dtype)
    want, _, _, _ = balance.forward(lg, k)
    bits = lg.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
    first = {}
    for i, pat in enumerate(NANS[dtype]):
        e = int(lg[i].float().argmin())
        bits[i, e] = pat
        first[i] = [e]
    bits[5, E - 1], bits[5, 1] = NANS[dtype][0], NANS[dtype][1]
    bits[6, E - 1], bits[6, 1] = NANS[dtype][2], NANS[dtype][0]
    first[5] = first[6] = [1, E - 1]
    idx, prob, counts, losses = m.moe_route_balance(lg.cuda(), k)
    torch.cuda.synchronize()
    idx, prob = idx.cpu(), prob.cpu()
    for t, ids in first.items():
        assert idx[t, :len(ids)].tolist() == ids, t
        assert torch.isnan(prob[t]).all(), t
    ok = [t for t in range(T) if t not in first]
    np.testing.assert_array_equal(idx[ok].numpy(), want[ok])
    assert torch.isfinite(prob[ok]).all() and torch.isnan(losses).all() and int(counts.sum()) == T * k
    # the gradient of such a token is NaN and stays with it
    d = m.moe_route_balance_bwd(lg.cuda(), idx.cuda(), prob.cuda(), counts, None, torch.ones(2, device="cuda")).cpu()
    assert torch.isnan(d[list(first)]).all() and torch.isfinite(d[ok]).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_nan_is_selected_ahead_of_infinity(dtype):
    m = need_gpu()
    nan, inf = float("nan"), float("inf")
    lg = torch.zeros((3, 20), dtype=dtype)
    lg[0, 2], lg[0, 9] = inf, nan
    lg[1, 0], lg[1, 3], lg[1, 18], lg[1, 19] = inf, nan, inf, -nan
    lg[2, 1], lg[2, 4], lg[2, 5] = inf, float(torch.finfo(dtype).max), inf
    idx, prob, _, losses = m.moe_route_balance(lg.cuda(), 4)
    torch.cuda.synchronize()
    assert idx.tolist() == [[9, 2, 0, 1], [3, 19, 0, 18], [1, 5, 4, 0]]
    assert torch.isnan(prob).all() and torch.isnan(losses).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_wide_rows_of_several_turns(dtype):
    """More tokens than the widest rows' kernels hold at once, forward (16384) and backward (20480)."""
    m = need_gpu()
    T, E, k = 20993, 131, 7
    lg, mask = _logits(T, E, "normal", dtype), _mask(T, True)
    idx, prob, counts, losses = m.moe_route_balance(lg.cuda(), k, token_mask=_gpu(mask))
    dprob = torch.from_numpy(np.random.default_rng(1).standard_normal((T, k)).astype(np.float32))
    dl = torch.tensor([0.8, 0.05])
    out = m.moe_route_balance_bwd(lg.cuda(), idx, prob, counts, dprob.cuda(), dl.cuda(), token_mask=_gpu(mask))
    torch.cuda.synchronize()
    ri, rp, rc, rl = balance.forward(lg, k, mask.numpy())
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    assert np.abs(prob.cpu().double().numpy() - rp).max() <= 40 * U
    assert (np.abs(losses.cpu().double().numpy() - rl) <= 80 * U * np.abs(rl)).all()
    want, mag = balance.backward(lg, ri, prob.cpu().numpy(), rc, dprob.numpy(), dl.numpy(), mask.numpy())
    err = np.abs(out.cpu().double().numpy() - want)
    tol = 48 * U * mag + np.abs(want) * float(torch.finfo(dtype).eps) / 2 + 1e-37
    assert (err <= tol).all(), float((err / tol).max())

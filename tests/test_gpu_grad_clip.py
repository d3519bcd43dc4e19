"""GPU parity of the global gradient norm and clipping against the fp64 oracle.

Tolerances, u = 2^-24: sums in 64 bits of exact squares, within n 2^-53 of themselves (1e-10 here); the norm and the
factor are one rounding each, the product another: an fp32 result within 3 u of itself, a bf16 one half a step more.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, need_gpu
from oracle import norm

U = 2.0 ** -24
F, B = torch.float32, torch.bfloat16


def _grads(sizes, dtypes, seed=0, scale=0.01):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(d) for n, d in zip(sizes, dtypes)]


def _np(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def _check(out, want, dtype):
    got = _np(out)
    tol = (3 * U + (float(torch.finfo(dtype).eps) / 2 if dtype == B else 0)) * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want) <= tol).all()


LISTS = [[1], [0, 3], [7, 0, 0, 65536], [32768], [32769, 1, 2, 3], [100003, 5, 77777], [3] * 300, [1000] * 129, [128, 1 << 20],
         list(range(1, 200)), [9] * 217, [2] * 313, [8193] * 433]


@gpu
@pytest.mark.parametrize("out", ["in place", "f32", "bf16"])
@pytest.mark.parametrize("kinds", ["f32", "bf16", "both"])
@pytest.mark.parametrize("i", range(len(LISTS)))
def test_norm_and_clip(i, kinds, out):
    m = need_gpu()
    sizes = LISTS[i]
    dt = [F if kinds == "f32" or (kinds == "both" and j % 3) else B for j in range(len(sizes))]
    g = _grads(sizes, dt, seed=i)
    ref = [_np(t) for t in g]
    full = float(np.sqrt(sum((r * r).sum() for r in ref)))
    for limit in (0.3 * full, 2 * full, float("inf"), 0.0):
        gg = [t.cuda() for t in g]
        od = dt if out == "in place" else [F if out == "f32" else B] * len(g)
        to = None if out == "in place" else [torch.empty(t.shape, dtype=d, device="cuda") for t, d in zip(g, od)]
        sq = m.moe_grad_sumsq(gg)
        n = m.moe_grad_clip(gg, limit, out=to)
        torch.cuda.synchronize()
        assert sq.dtype == torch.float64 and n.dtype == F and n.shape == (1,)
        assert abs(float(sq) - full ** 2) <= 1e-10 * full ** 2
        wn, want = norm.clip(ref, limit)
        assert abs(float(n) - wn) <= 2 * U * wn
        for o, w, d, t, before in zip(gg if to is None else to, want, od, gg, g):
            _check(o, w, d)
            if to is not None:
                assert torch.equal(t.cpu(), before)              # the gradients stay


@gpu
def test_a_table_keeps_and_the_norm_of_other_ranks():
    m = need_gpu()
    g = [t.cuda() for t in _grads([1000, 33, 70000], [F, B, F])]
    bucket = torch.zeros(71033, device="cuda")
    table = m.GradTable(g, list(bucket.split([1000, 33, 70000])))
    assert len(table) == 3
    sq = m.moe_grad_sumsq(table)
    total = sq * 5.5
    n = m.moe_grad_clip(table, 0.1, sumsq=total)
    torch.cuda.synchronize()
    wn, want = norm.clip([_np(t) for t in g], 0.1, float(total))
    assert abs(float(n) - wn) <= 2 * U * wn
    _check(bucket, np.concatenate(want), F)
    for t in g:                                                  # new values in the same places
        t.mul_(2)
    n2 = m.moe_grad_clip(table, 0.1)
    torch.cuda.synchronize()
    wn, want = norm.clip([_np(t) for t in g], 0.1)
    assert abs(float(n2) - wn) <= 2 * U * wn
    _check(bucket, np.concatenate(want), F)


@gpu
def test_values_at_odd_addresses():
    """Views of buckets that begin anywhere, input and output differently, and what lies between them stays."""
    m = need_gpu()
    g = torch.Generator().manual_seed(1)
    for di, do in ((F, F), (B, B), (F, B), (B, F)):
        a = (torch.randn(50000, generator=g) * 0.01).to(di).cuda()
        b = torch.full((50000,), 9.0, dtype=do, device="cuda")
        spans = [(1, 2), (5, 8), (13, 14), (101, 9000), (10003, 20001), (20002, 45001)]
        ins = [a[lo:hi] for lo, hi in spans]
        outs = [b[lo + 3:hi + 3] for lo, hi in spans]
        n = m.moe_grad_clip(ins, 0.2, out=outs)
        torch.cuda.synchronize()
        wn, want = norm.clip([_np(t) for t in ins], 0.2)
        assert abs(float(n) - wn) <= 2 * U * wn
        for o, w in zip(outs, want):
            _check(o, w, do)
        keep = torch.ones(50000, dtype=torch.bool)
        for lo, hi in spans:
            keep[lo + 3:hi + 3] = False
        assert (b.cpu()[keep] == 9).all()


@gpu
def test_large_and_small_values():
    """Squares past fp32's range either way."""
    m = need_gpu()
    for v in (1e30, 1e-30):
        g = [torch.full((1000,), v, device="cuda"), torch.full((24,), v, device="cuda", dtype=B)]
        ref = [_np(t) for t in g]
        sq = m.moe_grad_sumsq(g)
        want = sum((r * r).sum() for r in ref)
        assert abs(float(sq) - want) <= 1e-10 * want
        n = m.moe_grad_clip(g, 1.0)
        torch.cuda.synchronize()
        wn, out = norm.clip(ref, 1.0)
        assert abs(float(n) - wn) <= 2 * U * wn
        for t, w in zip(g, out):
            _check(t, w, t.dtype)


@gpu
def test_not_finite():
    m = need_gpu()
    g = [torch.ones(500, device="cuda"), torch.ones(3, device="cuda")]
    g[1][1] = float("inf")
    n = m.moe_grad_clip(g, 1.0)
    assert torch.isinf(n).all() and not g[0].any() and torch.isnan(g[1][1]) and float(g[1][0]) == 0
    g = [torch.ones(500, device="cuda"), torch.ones(3, device="cuda")]
    g[1][1] = float("nan")
    n = m.moe_grad_clip(g, 1.0)
    assert torch.isnan(n).all() and torch.isnan(g[0]).all()
    g = [torch.ones(5, device="cuda")]
    g[0][1] = float("inf")
    n = m.moe_grad_clip(g, float("inf"))
    assert torch.isinf(n).all() and float(g[0][0]) == 1 and torch.isinf(g[0][1])
    empty = torch.empty(0, device="cuda")
    n = m.moe_grad_clip([empty, empty], 1.0)
    assert float(n) == 0 and float(m.moe_grad_sumsq([empty])) == 0


@gpu
def test_streams_graphs_and_determinism():
    m = need_gpu()
    g = [t.cuda() for t in _grads([300000, 17, 4096], [F, B, F])]
    h = [t.cuda() for t in _grads([3] * 140, [B] * 140, seed=5)]
    og, oh = [torch.empty_like(t) for t in g], [torch.empty_like(t) for t in h]
    tg, th = m.GradTable(g, og), m.GradTable(h, oh)
    want = [m.moe_grad_clip(tg, 0.5)] + [t.clone() for t in og]
    want2 = [m.moe_grad_clip(th, 0.05)] + [t.clone() for t in oh]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        n1 = m.moe_grad_clip(tg, 0.5)
    with torch.cuda.graph(g2):
        n2 = m.moe_grad_clip(th, 0.05)
    for _ in range(3):
        for t in og + oh:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        m.moe_grad_sumsq(th)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([n1] + og, want))
        assert all(torch.equal(a, b) for a, b in zip([n2] + oh, want2))


@gpu
def test_refusals_on_the_gpu():
    m = need_gpu()
    a = torch.zeros(100, device="cuda")
    with pytest.raises(TypeError):
        m.moe_grad_sumsq([a, a.half()])
    with pytest.raises(TypeError):
        m.moe_grad_sumsq([a, torch.zeros(3)])
    with pytest.raises(ValueError):
        m.moe_grad_sumsq([a[::2]])
    with pytest.raises(ValueError):
        m.moe_grad_clip([a], 1.0, out=[torch.zeros(99, device="cuda")])
    with pytest.raises(ValueError):
        m.moe_grad_clip([a], 1.0, out=[a, a])
    with pytest.raises(ValueError):
        m.moe_grad_clip(m.GradTable([a]), 1.0, out=[a])
    with pytest.raises(TypeError):
        m.moe_grad_clip([a], 1.0, sumsq=torch.zeros(1, device="cuda"))
    for grads, out in (([a, a], None), ([a[:60], a[40:]], None), ([a[:60]], [a[30:90]])):
        with pytest.raises(m.MoeError):
            m.moe_grad_clip(grads, 1.0, out=out)
    with pytest.raises(m.MoeError):
        m.moe_grad_clip([a], -1.0)
    with pytest.raises(m.MoeError):
        m.moe_grad_clip([a], float("nan"))


@gpu
def test_a_norm_that_is_nan_shows_without_a_limit():
    """max_norm infinite: nothing is scaled, but a NaN norm makes every value NaN, as with any other limit."""
    m = need_gpu()
    nan, inf = float("nan"), float("inf")
    for dtype in (F, B):
        g = [torch.ones(9000, device="cuda", dtype=dtype), torch.ones(3, device="cuda")]
        g[1][1] = nan
        to = [torch.zeros(9000, device="cuda"), torch.zeros(3, device="cuda", dtype=B)]
        n = m.moe_grad_clip(g, inf, out=to)
        assert torch.isnan(n).all() and all(torch.isnan(t).all() for t in to)
        n = m.moe_grad_clip(g, inf)
        assert torch.isnan(n).all() and all(torch.isnan(t).all() for t in g)
    for limit in (inf, 1.0):
        g = [torch.ones(500, device="cuda")]
        n = m.moe_grad_clip(g, limit, sumsq=torch.full((1,), nan, device="cuda", dtype=torch.float64))
        assert torch.isnan(n).all() and torch.isnan(g[0]).all()
    g = [torch.ones(500, device="cuda")]
    n = m.moe_grad_clip(g, inf, sumsq=torch.full((1,), inf, device="cuda", dtype=torch.float64))
    assert torch.isinf(n).all() and (g[0] == 1).all()
    n = m.moe_grad_clip(g, 1.0, sumsq=torch.full((1,), inf, device="cuda", dtype=torch.float64))
    assert torch.isinf(n).all() and not g[0].any()


@gpu
def test_tensors_that_end_where_the_norm_and_the_sum_begin():
    """Beside one another in one piece of memory; a workspace that is not used may be anywhere.  Over one another: refused."""
    m = need_gpu()
    lib = m.load()
    from mixture_experts_grouped_permute_amd import _lib as L
    flat = torch.zeros(64, dtype=torch.float64, device="cuda")
    f32 = flat.view(F)
    g, sumsq, norm_at = f32[:20], flat[10:11], f32[22:23]
    g.fill_(2.0)
    table = m.GradTable([g])
    need = lib.moe_grad_sumsq_workspace(table._at[1], 1)
    ptrs, numel, kinds, outs, okinds = table._at
    def call(sum_at, norm_to, ws, wbytes):
        st = lib.moe_grad_clip(ptrs, numel, kinds, 1, outs, okinds, sum_at, 1.0, norm_to, ws, wbytes, L._stream(flat.device))
        torch.cuda.synchronize()
        return st
    sumsq.fill_(4.0)
    assert call(sumsq.data_ptr(), norm_at.data_ptr(), f32[4:].data_ptr(), need) == 0
    assert float(norm_at) == 2.0 and (g - 1.0).abs().max() <= 1e-6 and float(sumsq) == 4.0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert call(None, norm_at.data_ptr(), ws.data_ptr(), need) == 0
    assert abs(float(norm_at) - 20 ** 0.5) <= 1e-5
    for bad in ((sumsq.data_ptr(), sumsq.data_ptr() + 4, None, 0), (sumsq.data_ptr(), f32[19:].data_ptr(), None, 0),
                (g.data_ptr(), norm_at.data_ptr(), None, 0), (None, ws.data_ptr() + 8, ws.data_ptr(), need)):
        assert call(*bad) == L.MOE_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("kinds,out", [("f32", "in place"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "in place"),
                                       ("bf16", "f32"), ("both", "in place"), ("both", "bf16")])
def test_more_than_the_caches_hold(kinds, out):
    """Over 256 MB of gradients go past the caches: views at odd addresses, with tails and single values among them.  The
    64-bit sum over 7e7 values (1e-10 of itself) and the products on the GPU, by elementary operations."""
    m = need_gpu()
    wide = {"f32": 33_000_000, "bf16": 66_000_000, "both": 44_000_000}[kinds]
    sizes = [wide + 5, 1, 8191, wide + 8192, 8193, 7]
    dt = [F if kinds == "f32" or (kinds == "both" and i % 2 == 0) else B for i in range(6)]
    od = dt if out == "in place" else [F if out == "f32" else B] * 6
    gen = torch.Generator(device="cuda").manual_seed(len(kinds) + len(out))
    g, to = [], []
    for i, n in enumerate(sizes):
        flat = (torch.randn(n + 8, generator=gen, device="cuda") * 0.01).to(dt[i])
        g.append(flat[1 + i:1 + i + n])
        to.append(torch.full((n + 8,), 9.0, dtype=od[i], device="cuda")[3:3 + n] if out != "in place" else None)
    assert sum(t.numel() * t.element_size() for t in g) > 256e6
    before = [t.clone() for t in g]
    full = float(torch.stack([(t.double() * t.double()).sum() for t in g]).sum()) ** 0.5
    assert abs(float(m.moe_grad_sumsq(g)) - full ** 2) <= 1e-10 * full ** 2
    for limit in (2 * full, 0.3 * full):
        n = m.moe_grad_clip(g, limit, out=None if out == "in place" else to)
        torch.cuda.synchronize()
        assert abs(float(n) - full) <= 2 * U * full
        c = min(1.0, limit / (full + 1e-6))
        for o, d, b, t in zip(g if out == "in place" else to, od, before, g):
            want = b.double() * c
            tol = (3 * U + (float(torch.finfo(d).eps) / 2 if d == B else 0)) * want.abs() + 2.0 ** -133
            assert bool(((o.double() - want).abs() <= tol).all())
            assert out == "in place" or torch.equal(t, b)
        if out != "in place":
            for o, d in zip(to, od):                                  # (what lies around the views stays)
                whole = torch.empty(0, dtype=d, device="cuda").set_(o.untyped_storage())
                assert bool((whole[:3] == 9).all()) and bool((whole[3 + o.numel():] == 9).all())

"""GPU parity of the residual RMS norm (moe_add_rmsnorm and its gradient) against the fp64 oracle.

Tolerances, u = 2^-24.  The sum s is one fp32 addition rounded once: equal bit for bit to torch's.  The sum of squares
adds at most 128 values of a lane in turn and 10 levels of lanes: within 140 u of itself, its root 70 u; with the
division, the root and three products 80 u of y, and half an output step.  The gradient's mean is such a sum of terms
of either sign, within 140 u of the sum of their magnitudes, times factors within 80 u: 240 u of all terms' magnitudes.
dweight adds at most T terms in fp32, each within 80 u: (T + 100) u of the sum of their magnitudes.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, log, need_gpu
from oracle import norm

U = 2.0 ** -24
F, B = torch.float32, torch.bfloat16


def _x(T, H, dtype, seed):
    g = np.random.default_rng(seed + 3 * T + H)
    return torch.from_numpy((g.standard_normal((T, H)) * np.exp(0.7 * g.standard_normal(H))).astype(np.float32)).to(dtype)


def _w(H, dtype):
    return torch.from_numpy((1 + 0.1 * np.random.default_rng(H).standard_normal(H)).astype(np.float32)).to(dtype)


def _np(t):
    return t.detach().cpu().double().numpy()


def _half(dtype):
    return float(torch.finfo(dtype).eps) / 2


SHAPES = [(1, 1), (1, 7), (2, 64), (3, 128), (1, 4096), (5, 255), (4, 257), (300, 96), (7, 1003), (33, 1024), (130, 2048),
          (2, 8192), (3, 16384), (1, 32768), (2, 30001), (5, 8194), (1000, 130), (17, 4097), (9, 6016), (700, 640)]


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(B, B), (B, F), (F, F)], ids=["bf16", "bf16-w32", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_and_gradient(T, H, dtype, wdtype):
    m = need_gpu()
    log(f"norm {T} x {H} {dtype} {wdtype}")
    x, r, w = _x(T, H, dtype, 0), _x(T, H, dtype, 1), _w(H, wdtype)
    xs, rs, ws = x.cuda(), r.cuda(), w.cuda()
    for res in (None, rs):
        y, s, q, scales = m.moe_add_rmsnorm(xs, ws, residual=res, eps=1e-6)
        torch.cuda.synchronize()
        assert q is None and scales is None and y.dtype == dtype
        want_s = x if res is None else (x.float() + r.float()).to(dtype)
        assert (s is xs) if res is None else torch.equal(s.cpu(), want_s)
        want = norm.forward(want_s, w, 1e-6)
        err = np.abs(_np(y) - want)
        assert (err <= (80 * U + _half(dtype)) * np.abs(want) + 1e-38).all(), float((err / np.abs(want)).max())
    dy, ds = _x(T, H, dtype, 2), _x(T, H, dtype, 3)
    for d in (None, ds):
        dx, dw = m.moe_add_rmsnorm_bwd(dy.cuda(), s, ws, ds=None if d is None else d.cuda(), eps=1e-6)
        torch.cuda.synchronize()
        assert dx.dtype == dtype and dw.dtype == F
        rx, rw, mag, wmag = norm.backward(dy, want_s, w, 1e-6, d)
        err = np.abs(_np(dx) - rx)
        tol = 240 * U * mag + _half(dtype) * np.abs(rx) + 1e-38
        assert (err <= tol).all(), float((err / tol).max())
        err = np.abs(_np(dw) - rw)
        assert (err <= (T + 100) * U * wmag + 1e-38).all(), float((err / wmag).max() / U)


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(B, B), (B, F), (F, F)], ids=["bf16", "bf16-w32", "f32"])
@pytest.mark.parametrize("T,H", [(1, 128), (1, 4096), (3, 256), (50, 1408), (300, 2048), (37, 640), (2, 16384), (1, 32768),
                                 (129, 1152)])
def test_codes(T, H, dtype, wdtype):
    m = need_gpu()
    x, r, w = _x(T, H, dtype, 0), _x(T, H, dtype, 1), _w(H, wdtype)
    x[T // 2, :128] = 0
    r[T // 2, :128] = 0                           # a block of zeros
    xs, rs, ws = x.cuda(), r.cuda(), w.cuda()
    for res in (None, rs):
        y, s, q, scales = m.moe_add_rmsnorm(xs, ws, residual=res, codes=True)
        none, s2, q2, scales2 = m.moe_add_rmsnorm(xs, ws, residual=res, y=False, codes=True)
        y3, _, _, _ = m.moe_add_rmsnorm(xs, ws, residual=res)
        torch.cuda.synchronize()
        assert none is None and torch.equal(q, q2) and torch.equal(scales, scales2) and torch.equal(y, y3)
        assert torch.equal(s, s2)
        if dtype == F:                            # y is not rounded then: the quantizer's own result
            cq, cs = m.fp8_block_quantize(y)
            assert torch.equal(cq, q) and torch.equal(cs, scales)
        want = norm.forward(s.cpu(), w, 1e-6)
        amax = np.abs(want).reshape(T, H // 128, 128).max(axis=2).T
        d = np.where(amax > 0, amax / 448, 1.0)
        assert (np.abs(_np(scales) - d) <= 90 * U * d).all()
        got = _np(q.view(torch.float8_e4m3fn)).reshape(T, H // 128, 128) * _np(scales).T[:, :, None]
        # half a step: 2^-4 of a normal code, 2^-10 of the scale under 2^-6; the value itself within 90 u
        tol = np.maximum(np.abs(want).reshape(got.shape) * (2.0 ** -4 + 200 * U), d.T[:, :, None] * 2.0 ** -10 * (1 + 1e-4))
        assert (np.abs(got - want.reshape(got.shape)) <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", [B, F], ids=["bf16", "f32"])
def test_sum_in_place_and_gradient_in_place(dtype):
    m = need_gpu()
    for T, H in ((1, 4096), (70, 1003), (19, 2048), (3, 20000)):
        x, r, w = _x(T, H, dtype, 0).cuda(), _x(T, H, dtype, 1).cuda(), _w(H, dtype).cuda()
        want = m.moe_add_rmsnorm(x, w, residual=r, codes=H % 128 == 0)
        a, b = x.clone(), r.clone()
        for out, args in ((a, (a, r)), (b, (x, b))):
            got = m.moe_add_rmsnorm(args[0], w, residual=args[1], codes=H % 128 == 0, sum_out=out)
            torch.cuda.synchronize()
            assert got[1] is out
            for g, h in zip(got, want):
                assert (g is None and h is None) or torch.equal(g, h)


@gpu
@pytest.mark.parametrize("dtype", [B, F], ids=["bf16", "f32"])
def test_gradient_over_the_residuals_own(dtype):
    """dx written over dsum, as the C entry point allows."""
    m = need_gpu()
    from mixture_experts_grouped_permute_amd import _lib as L
    lib = m.load()
    # (10243, 20483: the last, moved-back piece of a row is a wave's first)
    for T, H in ((1, 4096), (3, 5), (600, 255), (40, 2048), (9, 30001), (700, 8192), (40, 10243), (40, 20483), (600, 10243),
                 (600, 20483)):
        dy, s, ds = (_x(T, H, dtype, i).cuda() for i in range(3))
        w = _w(H, dtype).cuda()
        want, wdw = m.moe_add_rmsnorm_bwd(dy, s, w, ds=ds)
        dx, dw = ds.clone(), torch.empty(H, device="cuda")
        ws = torch.empty(lib.moe_add_rmsnorm_bwd_workspace(T, H), dtype=torch.uint8, device="cuda")
        io = L._io(dy)
        st = lib.moe_add_rmsnorm_bwd(dy.data_ptr(), s.data_ptr(), dx.data_ptr(), io, w.data_ptr(), io, T, H, 1e-6,
                                     dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel(), L._stream(dy.device))
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(dx, want) and torch.equal(dw, wdw)


@gpu
def test_more_rows_than_a_launch_takes():
    m = need_gpu()
    T, H = (1 << 27) + 3, 8
    x = torch.ones((T, H), dtype=B, device="cuda")
    x[0], x[-1], x[-4] = _x(1, H, B, 0).cuda(), _x(1, H, B, 1).cuda(), _x(1, H, B, 2).cuda()
    w = _w(H, B).cuda()
    y, _, _, _ = m.moe_add_rmsnorm(x, w)
    dx, dw = m.moe_add_rmsnorm_bwd(x, x, w)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, T // 2, T - 4, T - 3, T - 2, T - 1], device="cuda")
    want = norm.forward(x[at].cpu(), w.cpu(), 1e-6)
    assert (np.abs(_np(y[at]) - want) <= (80 * U + _half(B)) * np.abs(want)).all()
    rx, _, mag, _ = norm.backward(x[at].cpu(), x[at].cpu(), w.cpu(), 1e-6)
    assert (np.abs(_np(dx[at]) - rx) <= 240 * U * mag + _half(B) * np.abs(rx) + 1e-38).all()


@gpu
def test_zero_rows_infinities_and_nan():
    m = need_gpu()
    for dtype in (B, F):
        x = _x(6, 256, dtype, 0)
        x[0] = 0
        x[1, 5], x[2, 9], x[3, 200] = float("nan"), float("inf"), -float("inf")
        w = _w(256, dtype)
        y, s, q, scales = m.moe_add_rmsnorm(x.cuda(), w.cuda(), eps=0.0, codes=True)
        torch.cuda.synchronize()
        want = norm.forward(x[4:], w, 0.0)
        assert (np.abs(_np(y)[4:] - want) <= (80 * U + _half(dtype)) * np.abs(want)).all()
        assert torch.isnan(y[0]).all() and torch.isnan(y[1]).all()          # 0 / 0, as the formula has it
        ref = torch.tensor([float("inf")]) * 0
        assert torch.isnan(ref).all() and torch.isnan(y[2, 9]) and float(y[2, 8]) == 0 and torch.isnan(y[3, 200])
        y, _, q, scales = m.moe_add_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, codes=True)
        torch.cuda.synchronize()
        assert not y[0].any() and not (q[0] & 0x7F).any() and (scales[:, 0] == 1).all()
        assert torch.isfinite(scales[:, 4:]).all() and torch.isnan(scales[:, 1]).all()


@gpu
def test_rows_at_the_ends_stay_apart():
    """Tensors inside larger ones, at odd places where only the type's alignment is asked for: nothing else changes."""
    m = need_gpu()
    for dtype, T, H in ((B, 5, 1001), (F, 3, 515), (B, 4, 1024)):
        def inside(t, shift):
            flat = torch.full((t.numel() + 64,), 7.0, dtype=dtype, device="cuda")
            v = flat[shift:shift + t.numel()].view(t.shape)
            v.copy_(t)
            return flat, v
        x, r, w = _x(T, H, dtype, 0), _x(T, H, dtype, 1), _w(H, dtype)
        (fx, xv), (fr, rv), (fw, wv) = inside(x, 1), inside(r, 3), inside(w, 5)
        fo, ov = inside(torch.zeros_like(x), 9)
        y, s, _, _ = m.moe_add_rmsnorm(xv, wv, residual=rv, sum_out=ov)
        y2, s2, _, _ = m.moe_add_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda())
        dx, dw = m.moe_add_rmsnorm_bwd(xv, rv, wv, ds=ov)
        dx2, dw2 = m.moe_add_rmsnorm_bwd(x.cuda(), r.cuda(), w.cuda(), ds=s2)
        torch.cuda.synchronize()
        want = norm.forward(s.cpu(), w, 1e-6)
        assert torch.equal(s, s2)
        for a, b in ((y, y2), (dx, dx2), (dw, dw2)):
            a, b = _np(a), _np(b)
            assert (np.abs(a - b) <= 2 * (1000 * U + _half(dtype)) * np.abs(b).max()).all()
        assert (np.abs(_np(y) - want) <= (80 * U + _half(dtype)) * np.abs(want)).all()
        assert (fo[:9] == 7).all() and (fo[9 + T * H:] == 7).all()


@gpu
def test_gradient_against_differences():
    """The kernels' own outputs moved by a step: fp32 in, so differences carry about 1e-3."""
    m = need_gpu()
    g = torch.Generator().manual_seed(4)
    s, w = torch.randn((3, 48), generator=g).cuda(), (1 + 0.1 * torch.randn(48, generator=g)).cuda()
    dy = torch.randn((3, 48), generator=g).cuda()
    dx, dw = m.moe_add_rmsnorm_bwd(dy, s, w)
    h = 1e-2
    def value(a, b):
        return float((m.moe_add_rmsnorm(a, b)[0].double() * dy.double()).sum())
    for t, i in ((0, 0), (1, 17), (2, 47)):
        a = s.clone(); a[t, i] += h
        b = s.clone(); b[t, i] -= h
        # h^2 / 6 of a third derivative of order 1, and 48 x 3 values' rounding 1e-6 over 2 h
        assert abs((value(a, w) - value(b, w)) / (2 * h) - float(dx[t, i])) <= 1e-3
        a = w.clone(); a[i] += h
        b = w.clone(); b[i] -= h
        assert abs((value(s, a) - value(s, b)) / (2 * h) - float(dw[i])) <= 1e-3


@gpu
def test_many_rows_and_determinism():
    m = need_gpu()
    for T, H, dtype in ((20011, 72, F), (9001, 384, B)):
        x, w, dy = _x(T, H, dtype, 0), _w(H, dtype), _x(T, H, dtype, 1)
        y, _, _, _ = m.moe_add_rmsnorm(x.cuda(), w.cuda())
        dx, dw = m.moe_add_rmsnorm_bwd(dy.cuda(), x.cuda(), w.cuda())
        dx2, dw2 = m.moe_add_rmsnorm_bwd(dy.cuda(), x.cuda(), w.cuda())
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        want = norm.forward(x[-500:], w, 1e-6)
        assert (np.abs(_np(y[-500:]) - want) <= (80 * U + _half(dtype)) * np.abs(want)).all()
        xd, wd, dd = _np(x), _np(w), _np(dy)
        r = 1 / np.sqrt((xd * xd).mean(1, keepdims=True) + 1e-6)
        terms = dd * xd * r
        assert (np.abs(_np(dw) - terms.sum(0)) <= (T + 100) * U * np.abs(terms).sum(0)).all()
        # far below that bound: rounding of either sign, a few hundred u of the root of the squares' sum
        assert (np.abs(_np(dw) - terms.sum(0)) <= 300 * U * np.sqrt((terms ** 2).sum(0)) * np.sqrt(T) / 8).all()


@gpu
def test_streams_and_graphs():
    m = need_gpu()
    x, r, w = _x(500, 1024, B, 0).cuda(), _x(500, 1024, B, 1).cuda(), _w(1024, B).cuda()
    x2, w2 = _x(300, 1001, F, 0).cuda(), _w(1001, F).cuda()

    def one():
        y, s, q, sc = m.moe_add_rmsnorm(x, w, residual=r, codes=True)
        return (y, s, q, sc) + m.moe_add_rmsnorm_bwd(y, s, w, ds=x)

    def two():
        y, s, _, _ = m.moe_add_rmsnorm(x2, w2)
        return (y,) + m.moe_add_rmsnorm_bwd(y, s, w2)

    want, want2 = one(), two()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s1):
        a = one()
    with torch.cuda.stream(s2):
        b = two()
    torch.cuda.synchronize()
    for got, ref in ((a, want), (b, want2)):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
    with torch.cuda.graph(g1):
        a = one()
    with torch.cuda.graph(g2):
        b = two()
    for _ in range(3):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        two()
        torch.cuda.synchronize()
        for got, ref in ((a, want), (b, want2)):
            assert all(torch.equal(p, q) for p, q in zip(got, ref))


@gpu
def test_refusals_on_the_gpu():
    m = need_gpu()
    x, w = torch.zeros((4, 256), device="cuda"), torch.ones(256, device="cuda")
    with pytest.raises(TypeError):
        m.moe_add_rmsnorm(x.half(), w)
    with pytest.raises(TypeError):
        m.moe_add_rmsnorm(x, w.bfloat16())
    with pytest.raises(TypeError):
        m.moe_add_rmsnorm(x, w, residual=x.bfloat16())
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w[:255])
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w, residual=x[:3])
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w, y=False)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x[:, :200].contiguous(), w[:200].contiguous(), codes=True)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm(x, w, sum_out=torch.empty_like(x))
    with pytest.raises(m.MoeError):
        m.moe_add_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(m.MoeError):
        m.moe_add_rmsnorm(torch.zeros((0, 256), device="cuda"), w)
    with pytest.raises(m.MoeError):
        m.moe_add_rmsnorm(torch.zeros((1, 40000), device="cuda"), torch.ones(40000, device="cuda"))
    with pytest.raises(m.MoeError):                       # codes want 16-byte rows
        m.moe_add_rmsnorm(torch.zeros(4 * 256 + 1, device="cuda")[1:].view(4, 256), w, codes=True)
    rows = torch.zeros((6, 256), device="cuda")
    with pytest.raises(m.MoeError):                       # the sum over a part of what is read
        m.moe_add_rmsnorm(rows[:4], w, residual=x, sum_out=rows[1:5])
    m.moe_add_rmsnorm(rows[:3], w, residual=x[:3], sum_out=rows[3:])    # (beside it)
    with pytest.raises(TypeError):
        m.moe_add_rmsnorm_bwd(x, x.bfloat16(), w)
    with pytest.raises(ValueError):
        m.moe_add_rmsnorm_bwd(x, x, w, ds=x[:2])


@gpu
@pytest.mark.parametrize("dtype", [B, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 64), (3, 8), (5, 255), (7, 128), (515, 130), (515, 96), (1001, 700), (513, 2048),
                                 (600, 1003), (2, 20483)])
def test_gradient_without_eps(T, H, dtype):
    """Places for rows that there are none of (a workgroup holds up to 16) leave the weight's gradient alone."""
    m = need_gpu()
    s, dy, w = _x(T, H, dtype, 0), _x(T, H, dtype, 1), _w(H, dtype)
    y, _, _, _ = m.moe_add_rmsnorm(s.cuda(), w.cuda(), eps=0.0)
    dx, dw = m.moe_add_rmsnorm_bwd(dy.cuda(), s.cuda(), w.cuda(), eps=0.0)
    torch.cuda.synchronize()
    want = norm.forward(s, w, 0.0)
    assert (np.abs(_np(y) - want) <= (80 * U + _half(dtype)) * np.abs(want) + 1e-38).all()
    rx, rw, mag, wmag = norm.backward(dy, s, w, 0.0)
    assert (np.abs(_np(dx) - rx) <= 240 * U * mag + _half(dtype) * np.abs(rx) + 1e-38).all()
    assert (np.abs(_np(dw) - rw) <= (T + 100) * U * wmag + 1e-38).all()


def _rows_on_gpu(T, H, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda")
    return x.mul_(torch.exp(0.7 * torch.randn(H, generator=g, device="cuda"))).to(dtype)


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(B, B), (B, F), (F, F)], ids=["bf16", "bf16-w32", "f32"])
@pytest.mark.parametrize("H", [104, 107, 248, 250, 509, 512, 1003, 1024, 2047, 2048, 4093, 4096, 8184, 8190, 16383, 16384, 30001,
                               32768])
def test_more_than_the_caches_hold(H, dtype, wdtype):
    """Results stored past the caches (402 MB forward, 604 backward), at each count of lanes a row, whole pieces and pieces
    that are moved back; dx apart from ds and over it.  The formulas in 64 bits on the GPU, by elementary operations.
    dweight: at least 256 workgroups share the rows, so a sum has at most T / 256 + 1 terms in turn, and 16 in LDS."""
    m = need_gpu()
    from mixture_experts_grouped_permute_amd import _lib as L
    lib = m.load()
    size = 2 if dtype == B else 4
    T = (576 << 20) // (4 * size * H) + 5
    log(f"norm {T} x {H} {dtype}")
    x, r, dy = (_rows_on_gpu(T, H, dtype, i) for i in range(3))
    w = _w(H, wdtype).cuda()
    kw = dict(residual=r, codes=H % 128 == 0)
    got = m.moe_add_rmsnorm(x, w, **kw)
    again = m.moe_add_rmsnorm(x, w, **kw)
    y, s, q, scales = got
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    if q is not None and dtype == F:
        cq, cs = m.fp8_block_quantize(y)
        assert torch.equal(cq, q) and torch.equal(cs, scales)
    dx, dw = m.moe_add_rmsnorm_bwd(dy, s, w, ds=r)
    over, dw2 = r.clone(), torch.empty(H, device="cuda")
    ws = torch.empty(lib.moe_add_rmsnorm_bwd_workspace(T, H), dtype=torch.uint8, device="cuda")
    st = lib.moe_add_rmsnorm_bwd(dy.data_ptr(), s.data_ptr(), over.data_ptr(), L._io(dy), w.data_ptr(), L._io(w), T, H, 1e-6,
                                 over.data_ptr(), dw2.data_ptr(), ws.data_ptr(), ws.numel(), L._stream(dy.device))
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(over, dx) and torch.equal(dw2, dw)
    w64, half = w.double(), _half(dtype)
    want_dw, mag_dw = torch.zeros(H, device="cuda", dtype=torch.float64), torch.zeros(H, device="cuda", dtype=torch.float64)
    step = max(1, (1 << 23) // H)
    for t in range(0, T, step):
        at = slice(t, min(t + step, T))
        s64, d64 = s[at].double(), dy[at].double()
        assert torch.equal(s[at], (x[at].float() + r[at].float()).to(dtype))
        rstd = 1 / torch.sqrt((s64 * s64).mean(1, keepdim=True) + 1e-6)
        xh = s64 * rstd
        want = xh * w64
        assert bool(((y[at].double() - want).abs() <= (80 * U + half) * want.abs() + 1e-38).all())
        gw = d64 * w64
        want = rstd * (gw - xh * (gw * xh).mean(1, keepdim=True)) + r[at].double()
        mag = rstd * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True)) + r[at].double().abs()
        assert bool(((dx[at].double() - want).abs() <= 240 * U * mag + half * want.abs() + 1e-38).all())
        want_dw += (d64 * xh).sum(0)
        mag_dw += (d64 * xh).abs().sum(0)
    assert bool(((dw.double() - want_dw).abs() <= (T / 256 + 120) * U * mag_dw).all())


@gpu
def test_weight_gradient_of_more_rows_than_a_launch_takes():
    """Terms of one sign, 16385 of them in turn by each of 512 x 16 places, 16 in LDS; each within 80 u.  (The oracle's sum
    over the 2^27 rows is in 64 bits.)"""
    m = need_gpu()
    T, H = (1 << 27) + 3, 8
    x, w = torch.empty((T, H), dtype=B, device="cuda"), _w(H, B).cuda()
    want = torch.zeros(H, device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda").manual_seed(3)
    step = 1 << 23
    for t in range(0, T, step):
        part = x[t:t + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        p64 = part.double()
        want += (p64 * p64 / torch.sqrt((p64 * p64).mean(1, keepdim=True) + 1e-6)).sum(0)
    _, dw = m.moe_add_rmsnorm_bwd(x, x, w)
    torch.cuda.synchronize()
    err = (dw.double() - want).abs() / want
    log(f"dweight off by {float(err.max()) / U:.0f} u")
    assert float(err.max()) <= (16385 + 16 + 100) * U

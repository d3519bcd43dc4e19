"""Host-side argument checks of grouped routing, the residual RMS norm and gradient clipping: every call here returns
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

P = 0x1000


@pytest.fixture(scope="module")
def lib():
    import mixture_experts_grouped_permute_amd as m
    return m.load()


def _codes():
    from mixture_experts_grouped_permute_amd import _lib as L
    return L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE


def _each(f, good, want, changes):
    assert f(*good) == want
    for at, bad, code in changes:
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)


def test_route_grouped_validation(lib):
    inv, uns, wsp = _codes()
    need = lib.moe_route_grouped_workspace(1000, 24)
    assert need > 0 and lib.moe_route_grouped_workspace(0, 8) == 0 and lib.moe_route_grouped_workspace(5, 257) == 0
    #        logits, type, bias, mask, T, E, k, score, G, kg, best, renorm, scale, idx, prob, counts, ws, bytes, stream
    good = [P, 0, None, None, 1000, 24, 4, 1, 4, 2, 2, 1, 1.0, P, P, P, P, need - 1, None]   # refused last, for its workspace
    nan, inf = float("nan"), float("inf")
    _each(lib.moe_route_grouped, good, wsp, [
        (0, None, inv), (1, 2, inv), (4, 0, inv), (4, 1 << 31, uns), (5, 0, inv), (5, 257, inv), (5, 25, inv), (6, 0, inv),
        (6, 17, inv), (6, 13, inv), (7, 2, inv), (7, -1, inv), (8, 0, inv), (8, 5, inv), (9, 0, inv), (9, 5, inv),
        (10, 0, inv), (10, 3, inv), (11, 2, inv), (12, 0.0, inv), (12, -1.0, inv), (12, nan, inv), (12, inf, inv),
        (13, None, inv), (14, None, inv), (16, None, wsp)])
    a = list(good)
    a[8], a[9], a[10] = 24, 5, 1
    assert lib.moe_route_grouped(*a) == uns                       # more groups than 16
    a[10] = 2
    assert lib.moe_route_grouped(*a) == inv                       # two best of groups of one
    a = list(good)
    a[3], a[15] = P, None
    assert lib.moe_route_grouped(*a) == inv                       # a mask without counts
    a = list(good)
    a[16], a[17] = P + 8, need
    assert lib.moe_route_grouped(*a) == uns


def test_route_grouped_bwd_validation(lib):
    inv, uns, _ = _codes()
    f = lib.moe_route_grouped_bwd
    good = [None, 0, 10, 8, 2, 1, 1, 1.0, P, P, P, P, None]
    assert f(*good) == inv
    good[0] = P
    for at, bad, code in ((1, 3, inv), (2, 0, inv), (2, 1 << 31, uns), (3, 0, inv), (4, 9, inv), (5, 2, inv), (6, 2, inv),
                          (7, 0.0, inv), (7, float("nan"), inv), (8, None, inv), (9, None, inv), (10, None, inv),
                          (11, None, inv)):
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)


def test_add_rmsnorm_validation(lib):
    inv, uns, _ = _codes()
    f = lib.moe_add_rmsnorm
    #       x, residual, type, weight, type, T, H, eps, sum, y, q, scales, stream
    good = [P, P, 1, P, 1, 8, 256, 1e-6, P, P, P, P, None]
    for at, bad, code in ((0, None, inv), (2, 2, inv), (3, None, inv), (4, 3, inv), (5, 0, inv), (6, 0, inv), (7, -1.0, inv),
                          (7, float("nan"), inv), (8, None, inv), (1, None, inv), (10, None, inv), (11, None, inv),
                          (5, 1 << 31, uns), (6, 32768 + 128, uns), (6, 200, uns), (0, P + 8, uns), (1, P + 8, uns),
                          (3, P + 2, uns), (8, P + 8, uns), (9, P + 8, uns), (10, P + 4, uns)):
        a = list(good)
        a[at] = bad
        assert f(*a) == code, (at, bad)
    a = list(good)
    a[9] = a[10] = a[11] = None
    assert f(*a) == inv                                           # no output
    a = list(good)
    a[2], a[4] = 0, 1
    assert f(*a) == uns                                           # fp32 activations, bf16 weight


def test_add_rmsnorm_bwd_validation(lib):
    inv, uns, wsp = _codes()
    need = lib.moe_add_rmsnorm_bwd_workspace(8, 200)
    assert need > 0 and lib.moe_add_rmsnorm_bwd_workspace(0, 8) == 0 and lib.moe_add_rmsnorm_bwd_workspace(8, 32769) == 0
    #       dy, s, dsum, type, weight, type, T, H, eps, dx, dw, ws, bytes, stream
    good = [P, P, None, 1, P, 0, 8, 200, 1e-6, P, P, P, need - 1, None]
    _each(lib.moe_add_rmsnorm_bwd, good, wsp, [
        (0, None, inv), (1, None, inv), (3, 2, inv), (4, None, inv), (5, 2, inv), (6, 0, inv), (7, 0, inv), (8, -1.0, inv),
        (9, None, inv), (10, None, inv), (11, None, wsp), (6, 1 << 31, uns), (7, 32769, uns)])
    a = list(good)
    a[11], a[12] = P + 4, need
    assert lib.moe_add_rmsnorm_bwd(*a) == uns


def test_the_norms_outputs_are_held_apart(lib):
    inv, _, _ = _codes()
    MB = 1 << 20
    T, H = 64, 256                                                # 32 KB in bf16, 64 in fp32
    x, r, w, s, y, q, d, ws = (MB * (i + 1) for i in range(8))
    ok = dict(x=x, r=r, w=w, s=s, y=y, q=q, d=d)
    for change in (dict(s=x + 16), dict(s=r - 16), dict(s=x + T * H * 2 - 16), dict(y=x), dict(y=r + 32), dict(s=y), dict(q=x),
                   dict(q=y + T * H), dict(d=q + T * H - 4), dict(w=s + 64), dict(d=w + H * 2 - 4), dict(s=x, y=x)):
        a = dict(ok, **change)
        assert lib.moe_add_rmsnorm(a["x"], a["r"], 1, a["w"], 1, T, H, 1e-6, a["s"], a["y"], a["q"], a["d"], None) == inv, change
    need = lib.moe_add_rmsnorm_bwd_workspace(T, H)
    ok = dict(dy=x, s=r, ds=s, w=w, dx=y, dw=q, ws=ws)
    for change in (dict(dx=x), dict(dx=r), dict(dx=s + 16), dict(dx=s - 4), dict(dw=w), dict(dw=y + 64), dict(ws=x + 16),
                   dict(dw=ws + need - 16), dict(ws=r - need + 16), dict(dx=s, dy=s)):
        a = dict(ok, **change)
        assert lib.moe_add_rmsnorm_bwd(a["dy"], a["s"], a["ds"], 0, a["w"], 0, T, H, 1e-6, a["dx"], a["dw"], a["ws"], need,
                                       None) == inv, change


def _arrays(ptrs, numel, kinds):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*kinds)


def test_grad_sumsq_validation(lib):
    inv, uns, wsp = _codes()
    g, numel, kinds = _arrays([P, None, 4 * P], [10, 0, 100], [0, 1, 1])
    need = lib.moe_grad_sumsq_workspace(numel, 3)
    assert need > 0 and lib.moe_grad_sumsq_workspace(numel, 0) == 0 and lib.moe_grad_sumsq_workspace(None, 3) == 0
    good = [g, numel, kinds, 3, P, P, need - 1, None]
    _each(lib.moe_grad_sumsq, good, wsp, [(0, None, inv), (1, None, inv), (2, None, inv), (3, 0, inv), (3, 65537, uns),
                                          (4, None, inv), (5, None, wsp)])
    for ptrs, n, k, code in (([P, None], [1, 1], [0, 0], inv), ([P, P], [1, -1], [0, 0], inv), ([P, P], [1, 1], [0, 2], inv),
                             ([P, P], [1, (1 << 35) + 1], [0, 0], uns)):
        a, b, c = _arrays(ptrs, n, k)
        assert lib.moe_grad_sumsq(a, b, c, 2, P, P, 1 << 30, None) == code
    assert lib.moe_grad_sumsq(g, numel, kinds, 3, P, P + 8, need, None) == uns


def _clip(lib, ptrs, numel, kinds, outs, okinds, *, sumsq=P, max_norm=1.0, norm=None, ws=None, wbytes=0):
    """(with norm None every call is refused: the others of the checks come first)"""
    g, n, k = _arrays(ptrs, numel, kinds)
    o, _, ok = _arrays(outs, numel, okinds)
    return lib.moe_grad_clip(g, n, k, len(ptrs), o, ok, sumsq, max_norm, norm, ws, wbytes, None)


def test_grad_clip_validation(lib):
    inv, uns, wsp = _codes()
    assert _clip(lib, [P], [4], [0], [P], [0]) == inv                             # no norm
    need = lib.moe_grad_sumsq_workspace((ctypes.c_int64 * 1)(4), 1)               # its own sum takes a workspace
    assert _clip(lib, [P], [4], [0], [P], [0], sumsq=None, norm=P) == wsp
    assert _clip(lib, [P], [4], [0], [P], [0], sumsq=None, norm=P, ws=P, wbytes=need - 1) == wsp
    assert _clip(lib, [P], [4], [0], [P], [0], sumsq=None, norm=P, ws=P + 8, wbytes=need) == uns
    assert _clip(lib, [P], [4], [0], [P], [0], max_norm=-1.0, norm=P) == inv
    assert _clip(lib, [P], [4], [0], [P], [0], max_norm=float("nan"), norm=P) == inv
    assert _clip(lib, [P], [4], [0], [None], [0], norm=P) == inv
    assert _clip(lib, [P], [4], [0], [2 * P], [2], norm=P) == inv
    assert _clip(lib, [P], [(1 << 35) + 1], [0], [P], [0], norm=P) == uns
    assert _clip(lib, [1 << 47], [4], [0], [P], [0], norm=P) == uns               # no address of a process
    assert _clip(lib, [P], [4], [0], [(1 << 48) + P], [0], norm=P) == uns


def test_grad_clip_refuses_overlaps(lib):
    """Outputs that another value of the call shares memory with: workgroups take them in no order."""
    inv, _, _ = _codes()
    for ptrs, numel, kinds, outs, okinds in (
            ([P, P], [4, 4], [0, 0], [P, P], [0, 0]),                              # one gradient twice, in place
            ([P, P + 8], [4, 4], [0, 0], [P, P + 8], [0, 0]),                      # two that share values
            ([P], [4], [0], [P + 4], [0]),                                         # shifted onto itself
            ([P], [4], [1], [P], [0]),                                             # in place, of a wider type
            ([P], [4], [0], [P], [1]),                                             # and of a narrower one
            ([P, 2 * P], [4, 4], [0, 0], [2 * P, P], [0, 0]),                      # exchanged
            ([4 * P, P, 8 * P], [4, 4096, 4], [0, 0, 0], [16 * P, 32 * P, P + 400], [0, 0, 0]),
            ([P, 2 * P], [4, 4], [0, 0], [8 * P, 8 * P + 12], [0, 0])):            # outputs that share a value
        assert _clip(lib, ptrs, numel, kinds, outs, okinds, norm=P) == inv, (ptrs, outs)


def test_binding_refusals():
    import mixture_experts_grouped_permute_amd as m
    x, w = torch.zeros(4, 128), torch.ones(128)
    i4, f4 = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    for call in (lambda: m.moe_route_grouped(x, 2), lambda: m.moe_route_grouped_bwd(x, i4, f4, f4),
                 lambda: m.moe_add_rmsnorm(x, w), lambda: m.moe_add_rmsnorm_bwd(x, x, w), lambda: m.GradTable([x]),
                 lambda: m.moe_grad_sumsq([x]), lambda: m.moe_grad_clip([x], 1.0)):
        with pytest.raises(TypeError, match="GPU"):
            call()
    with pytest.raises(ValueError):
        m.GradTable([])
    with pytest.raises(ValueError):
        m.GradTable([x], [x, x])


def test_grad_clip_refuses_outputs_over_its_norm_sum_and_workspace(lib):
    """What the workgroups read their factor from, or leave the norm in, shares no memory with what others write."""
    inv, _, wsp = _codes()
    MB = 1 << 20
    need = lib.moe_grad_sumsq_workspace((ctypes.c_int64 * 2)(1000, 70000), 2)
    def call(sumsq, norm, ws, outs=(16 * MB, 20 * MB)):
        return _clip(lib, [MB, 4 * MB], [1000, 70000], [0, 1], outs, [0, 0], sumsq=sumsq, norm=norm, ws=ws, wbytes=need)
    for sumsq, norm, ws, outs in (
            (16 * MB + 8, 8 * MB, None, (16 * MB, 20 * MB)),                       # the sum in an output
            (20 * MB + 70000 * 4 - 8, 8 * MB, None, (16 * MB, 20 * MB)),
            (9 * MB, 16 * MB + 3996, None, (16 * MB, 20 * MB)),                    # the norm in an output, in a gradient
            (9 * MB, 4 * MB + 2 * 69998, None, (16 * MB, 20 * MB)),
            (9 * MB, 9 * MB + 4, None, (16 * MB, 20 * MB)),                        # the norm over the sum
            (MB + 400, 8 * MB, None, (MB, 20 * MB)),                               # in place
            (9 * MB, MB, None, (MB, 20 * MB)),
            (None, 8 * MB, 16 * MB + 3984, (16 * MB, 20 * MB)),                    # the workspace: in an output, in a gradient,
            (None, 8 * MB, MB - need + 16, (16 * MB, 20 * MB)),                    # over the norm
            (None, 8 * MB + need - 16, 8 * MB, (16 * MB, 20 * MB))):
        assert call(sumsq, norm, ws, outs) == inv, (sumsq, norm, ws, outs)
    assert call(None, 16 * MB, None) == wsp

"""Host-side argument checks of the training router and the block-scaled FP8 entry points: every call
here returns before anything is enqueued (no GPU needed)."""
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


def test_route_balance_validation(lib):
    inv, _, wsp = _codes()
    need = lib.moe_route_balance_workspace(1000, 8)
    assert need > 0 and lib.moe_route_balance_workspace(0, 8) == 0 and lib.moe_route_balance_workspace(5, 257) == 0
    good = [P, 0, None, 1000, 8, 2, P, P, P, P, P, need - 1, None]      # refused last, for its workspace
    assert lib.moe_route_balance(*good) == wsp
    for at, bad in ((0, None), (1, 2), (3, 0), (4, 257), (5, 0), (5, 9), (5, 17), (6, None), (7, None), (8, None),
                    (9, None)):
        a = list(good)
        a[at] = bad
        assert lib.moe_route_balance(*a) == inv, at
    a = list(good)
    a[10] = None
    assert lib.moe_route_balance(*a) == wsp


def test_route_balance_bwd_validation(lib):
    inv, uns, _ = _codes()
    f = lib.moe_route_balance_bwd
    assert f(None, 0, None, 10, 8, 2, P, P, P, P, P, P, None) == inv
    assert f(P, 0, None, 10, 8, 2, None, P, P, P, P, P, None) == inv      # dprob without ids
    assert f(P, 0, None, 10, 8, 2, P, None, P, P, P, P, None) == inv
    assert f(P, 0, None, 10, 8, 2, P, P, None, P, P, P, None) == inv
    assert f(P, 0, None, 10, 8, 2, P, P, P, P, P, None, None) == inv
    assert f(P, 0, None, 10, 8, 9, P, P, P, P, P, P, None) == inv
    assert f(P, 0, None, 1 << 31, 8, 2, P, P, P, P, P, P, None) == uns


def test_fp8_block_quantize_validation(lib):
    inv, uns, _ = _codes()
    f = lib.fp8_block_quantize
    assert f(None, 1, 8, 128, 0, None, 0, P, P, None) == inv
    assert f(P, 1, 0, 128, 0, None, 0, P, P, None) == inv
    assert f(P, 2, 8, 128, 0, None, 0, P, P, None) == inv
    assert f(P, 1, 8, 128, 2, None, 0, P, P, None) == inv
    assert f(P, 1, 8, 192, 0, None, 0, P, P, None) == uns
    assert f(P + 8, 1, 8, 128, 0, None, 0, P, P, None) == uns             # alignment
    assert f(P, 1, 8, 128, 1, None, 2, P, P, None) == inv                 # two groups need offsets
    assert f(P, 1, 8, 128, 1, P, 257, P, P, None) == inv
    assert f(P, 1, 8, 24, 1, P, 2, P, P, None) == uns
    assert f(P, 1, 1 << 31, 128, 0, None, 0, P, P, None) == uns


def test_fp8_block_weights_validation(lib):
    inv, uns, _ = _codes()
    f = lib.fp8_block_quantize_weights
    tab = (ctypes.c_void_p * 2)(P, P)
    bad = (ctypes.c_void_p * 2)(P, None)
    assert f(tab, 0, 128, 128, 0, None, P, P, None) == inv
    assert f(bad, 2, 128, 128, 0, None, P, P, None) == inv
    assert f(tab, 2, 128, 128, 2, None, P, P, None) == inv
    assert f(tab, 2, 128, 144, 0, None, P, P, None) == uns
    assert f(tab, 2, 136, 128, 0, None, P, P, None) == uns
    assert f(tab, 2, 144, 128, 1, None, P, P, None) == uns
    assert f(tab, 2, 128, 136, 1, None, P, P, None) == uns
    assert f(tab, 2, 128, 128, 0, None, P + 4, P, None) == uns


def test_fp8_block_products_validation(lib):
    inv, uns, wsp = _codes()
    f = lib.fp8_block_grouped_gemm
    good = [P, P, P, P, P, 8, 128, 128, 2, 1, P, P, 1 << 30, None]
    for at, val, code in ((0, None, inv), (4, None, inv), (5, 0, inv), (8, 0, inv), (8, 257, inv), (9, 2, inv),
                          (10, None, inv), (7, 192, uns), (6, 136, uns), (0, P + 8, uns), (10, P + 8, uns),
                          (5, 1 << 31, uns), (6, 1 << 23, uns), (7, 1 << 24, uns)):
        a = list(good)
        a[at] = val
        assert f(*a) == code, (at, val)
    f = lib.fp8_block_grouped_wgrad
    for at, val, code in ((0, None, inv), (3, None, inv), (5, 0, inv), (9, 3, inv), (5, 136, uns), (6, 136, uns),
                          (7, 24, uns), (10, P + 4, uns), (5, 1 << 24, uns)):
        a = list(good)
        a[at] = val
        assert f(*a) == code, (at, val)


def test_fp8_block_products_workspace(lib):
    inv, uns, wsp = _codes()
    for f, size in ((lib.fp8_block_grouped_gemm, lib.fp8_block_grouped_gemm_workspace),
                    (lib.fp8_block_grouped_wgrad, lib.fp8_block_grouped_wgrad_workspace)):
        assert size(0, 128, 128, 1, 1) == 0 and size(8, 128, 128, 1, 2) == 0 and size(8, 128, 128, 0, 1) == 0
        n = size(8192, 512, 8192, 2, 1)
        assert n > 0
        a = [P, P, P, P, P, 8192, 512, 8192, 2, 1, P, P, n - 1, None]
        assert f(*a) == wsp
        a[11], a[12] = None, n
        assert f(*a) == wsp
        a[11] = P + 4
        assert f(*a) == uns


def test_binding_refuses_tensors_off_the_gpu():
    import mixture_experts_grouped_permute_amd as m
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    u8, f4, i4 = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        m.moe_route_balance(x, 2)
    with pytest.raises(TypeError):
        m.moe_route_balance_bwd(x, i4, f4, i4)
    with pytest.raises(TypeError):
        m.fp8_block_quantize(x)
    with pytest.raises(TypeError):
        m.fp8_block_quantize_weights(x[None])
    with pytest.raises(TypeError):
        m.fp8_block_grouped_gemm(u8, f4, u8[None], f4, i4)
    with pytest.raises(TypeError):
        m.fp8_block_grouped_wgrad(u8, f4, u8, f4, i4)


def _weights(compute, transposed, E=3, H=256, I=384):
    """Tensors of quantize_weights' shapes."""
    out = []
    for n, k in ((H, 2 * I), (I, H)) if transposed else ((2 * I, H), (H, I)):
        out.append(torch.zeros((E, n, k), dtype=torch.uint8))
        out.append({"mxfp8": torch.zeros((E, n, k // 32), dtype=torch.uint8), "fp8": torch.zeros(E),
                    "fp8_block": torch.zeros((E, n // 128, k // 128))}[compute])
    return tuple(out)


@pytest.mark.parametrize("compute", ["mxfp8", "fp8", "fp8_block"])
def test_cached_weights_of_another_precision_are_refused(compute):
    """Ahead of the library, which sees pointers only: the scales' sizes differ between the precisions."""
    import mixture_experts_grouped_permute_amd as m
    from mixture_experts_grouped_permute_amd import _lib as L
    T, H, I, E, k = 4, 256, 384, 3, 1
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    idx, prob = torch.zeros((T, k), dtype=torch.int32), torch.ones((T, k))
    w1, w2 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16), torch.zeros((E, H, I), dtype=torch.bfloat16)
    good = _weights(compute, False)
    L._cached(good, compute, False, E, H, I, x.device)
    wrong = [_weights(c, False) for c in ("mxfp8", "fp8", "fp8_block") if c != compute]
    if compute != "fp8":
        wrong.append(_weights(compute, True))
    wrong += [good[2:] + good[:2], good[:3], good[:1] + (good[1][1:],) + good[2:], tuple(t[:2].contiguous() for t in good),
              good[:3] + (good[3].double(),)]
    for w in wrong:
        with pytest.raises((TypeError, ValueError), match="cached weights"):
            m.moe_grouped_mlp_fwd(x, idx, prob, w1, w2, compute, w_quant=w)


@pytest.mark.parametrize("compute", ["mxfp8", "fp8_block"])
def test_cached_transposed_weights_of_another_form_are_refused(compute):
    import mixture_experts_grouped_permute_amd as m
    from mixture_experts_grouped_permute_amd import _lib as L
    T, H, I, E = 4, 256, 384, 3
    dy = torch.zeros((T, H), dtype=torch.bfloat16)
    w1, w2 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16), torch.zeros((E, H, I), dtype=torch.bfloat16)
    perm = {n: torch.zeros(c, dtype=torch.int32) for n, c in
            (("split_sizes", E), ("offsets", E + 1), ("row_id_map", T), ("src_index", T))}
    perm["prob_perm"] = torch.zeros(T)
    saved = {n: torch.zeros((T, c), dtype=torch.bfloat16) for n, c in (("x_perm", H), ("gu", 2 * I), ("h", I))}
    ctx = {"perm": perm, "saved": saved, "compute": compute, "E": E, "I": I}
    good = _weights(compute, True)
    L._cached(good, compute, True, E, H, I, dy.device)
    other = "mxfp8" if compute == "fp8_block" else "fp8_block"
    for w in (_weights(compute, False), _weights(other, True), good[2:] + good[:2], good[:2]):
        with pytest.raises((TypeError, ValueError), match="cached transposed weights"):
            m.moe_grouped_mlp_bwd(dy, ctx, w1, w2, w_quant_t=w)
    # square sizes (2 I = H): the second pair still tells the two forms apart
    for a, b in ((True, False), (False, True)):
        with pytest.raises(ValueError, match="cached"):
            L._cached(_weights(compute, a, H=256, I=128), compute, b, E, 256, 128, dy.device)


def test_stream_handles_without_the_private_accessor(monkeypatch):
    from types import SimpleNamespace
    from mixture_experts_grouped_permute_amd import _lib as L
    dev = torch.device("cuda", 1)
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: asked.append(d) or SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(L, "_raw_stream", None)
    assert L._stream(dev) == 7 and asked == [dev]
    monkeypatch.setattr(L, "_raw_stream", lambda index: 100 + index)
    assert L._stream(dev) == 101


def test_rows_past_one_launch_are_refused(lib):
    """2^32 threads or more: refused with the sizes, not by the launch."""
    _, uns, _ = _codes()
    f = lib.fp8_block_quantize
    for rows, cols in ((1 << 28, 128), ((1 << 27) + 1, 640), ((1 << 31) - 1, 512)):
        assert f(P, 1, rows, cols, 0, None, 0, P, P, None) == uns, (rows, cols)
    from mixture_experts_grouped_permute_amd._lib import FwdArgs
    tab = (ctypes.c_void_p * 2)(P, P)
    for T, want in ((1 << 28, False), ((1 << 28) - 16, True)):
        a = FwdArgs(T=T, H=128, I=128, E=2, k=1, compute=4, io_dtype=1, x=P, topk_idx=P, topk_prob=P, w1=tab, w2=tab,
                    out=P, split_sizes=P, offsets=P, row_id_map=P, src_index=P, prob_perm=P)
        assert (lib.moe_grouped_mlp_fwd_workspace(ctypes.byref(a)) > 0) == want, T


def test_products_of_few_rows_end_at_512(lib):
    """Products of few rows, which read the weights once for 16 rows of an expert and need no scratch, are
    bounded in rows as well as in rows an expert."""
    size = lib.fp8_block_grouped_gemm_workspace
    for R, E, few in ((512, 256, True), (513, 256, False), (2048, 256, False), (512, 64, True), (513, 64, False),
                      (16, 1, True), (17, 1, False), (64, 8, True), (65, 8, False)):
        assert (size(R, 512, 8192, E, 1) == 0) == few, (R, E)


def test_captured_calls_share_no_workspace(monkeypatch):
    """Eager calls of a stream share its buffer; a captured one has its own, which is not kept: two graphs captured
    on one stream may be replayed at once on two."""
    from types import SimpleNamespace
    from mixture_experts_grouped_permute_amd import _lib as L
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    ws, cpu = L._Workspace(), torch.device("cpu")
    a = ws.get(1000, cpu)
    assert ws.get(500, cpu) is a
    capturing[0] = True
    b, c = ws.get(500, cpu), ws.get(500, cpu)
    assert len({t.data_ptr() for t in (a, b, c)}) == 3
    assert ws.holds(a) and not ws.holds(b) and not ws.holds(c)
    capturing[0] = False
    assert ws.get(500, cpu) is a


def test_layer_refuses_codes_and_gradients_off_16_bytes(lib):
    """What the block-scaled products refuse by themselves."""
    _, uns, wsp = _codes()
    from mixture_experts_grouped_permute_amd._lib import BwdArgs, FwdArgs
    tab = (ctypes.c_void_p * 2)(P, P)
    f = dict(T=64, H=128, I=128, E=2, k=1, compute=4, io_dtype=1, x=P, topk_idx=P, topk_prob=P, w1=tab, w2=tab, out=P,
             split_sizes=P, offsets=P, row_id_map=P, src_index=P, prob_perm=P, w1q=P, w2q=P, w1_scale=P, w2_scale=P)
    for kw, want in (({}, wsp), (dict(w1q=P + 8), uns), (dict(w2q=P + 4), uns)):
        a = FwdArgs(**{**f, **kw})
        assert lib.moe_grouped_mlp_fwd(ctypes.byref(a), None) == want, kw
    b = dict(T=64, H=128, I=128, E=2, k=1, compute=4, io_dtype=1, dw_dtype=0, dy=P, w1=tab, w2=tab, split_sizes=P, offsets=P,
             row_id_map=P, src_index=P, prob_perm=P, saved_x_perm=P, saved_gu=P, saved_h=P, dx=P, dprob=P, dw1=tab, dw2=tab,
             w1tq=P, w1ts=P, w2tq=P, w2ts=P)
    off = (ctypes.c_void_p * 2)(P, P + 8)
    for kw, want in (({}, wsp), (dict(w1tq=P + 8), uns), (dict(w2tq=P + 4), uns), (dict(dw1=off), uns), (dict(dw2=off), uns)):
        a = BwdArgs(**{**b, **kw})
        assert lib.moe_grouped_mlp_bwd(ctypes.byref(a), None) == want, kw

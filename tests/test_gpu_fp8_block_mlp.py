"""GPU parity of the expert MLP with block-scaled FP8 operands (compute "fp8_block"), forward and
backward, and of a training step of router and experts together.

Normwise, at the E4M3 tolerance of the other 8-bit paths (2e-2): both sides round the same values to the
same formats, but fp32 and fp64 arithmetic ahead of a rounding may put a value on either side of a
border, one E4M3 step (2^-3 at most) apart.
"""
import numpy as np
import pytest
import torch

from gpu_util import MXFP8_TOL, cfg_small, gpu, inputs_with_counts, log, need_gpu, to_np
from moe_inputs import make_inputs
from oracle import balance, mlp

CASES = [
    # T, H, I, E, k, x dtype, counts
    (1, 128, 128, 1, 1, "bf16", None),
    (64, 256, 384, 4, 2, "bf16", None),
    (300, 128, 256, 8, 2, "f32", None),
    (257, 512, 640, 5, 3, "bf16", None),
    (300, 256, 128, 6, 1, "bf16", [0, 33, 0, 255, 12, 0]),
    (700, 384, 256, 3, 1, "f32", [600, 100, 0]),
    # few rows an expert, as in decoding
    (3, 256, 384, 8, 2, "bf16", None),
    (20, 128, 256, 16, 4, "f32", None),
    (100, 640, 1152, 16, 1, "bf16", [90] + [0] * 13 + [4, 6]),
]
IDS = [f"T{c[0]}-H{c[1]}-I{c[2]}-E{c[3]}-k{c[4]}-{c[5]}{'-counts' if c[6] else ''}" for c in CASES]


def _inputs(case):
    T, H, I, E, k, xd, counts = case
    cfg = cfg_small(T=T, H=H, I=I, E=E, k=k, x_dtype=xd, seed=40 + T)
    if counts is None:
        return cfg, make_inputs(cfg, with_dy=True)
    inp = inputs_with_counts(cfg, counts)
    full = make_inputs(cfg, with_dy=True)
    inp.dy = full.dy
    return cfg, inp


def _oracle(cfg, inp):
    fw = mlp.forward(inp.x, inp.topk_idx.numpy(), inp.topk_prob, inp.w1, inp.w2, "fp8_block", cfg.x_dtype)
    return fw, mlp.backward(fw, inp.x, inp.dy, inp.w1, inp.w2)


@gpu
@pytest.mark.parametrize("dw", [torch.float32, torch.bfloat16], ids=["dw-f32", "dw-bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward(case, dw):
    m = need_gpu()
    cfg, inp = _inputs(case)
    log(f"fp8_block mlp {case}")
    d = inp.to("cuda")
    out, ctx = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, "fp8_block", save_for_backward=True)
    dx, dprob, dw1, dw2 = m.moe_grouped_mlp_bwd(d.dy, ctx, d.w1, d.w2, dw_dtype=dw)
    torch.cuda.synchronize()
    fw, bw = _oracle(cfg, inp)
    errs = {n: mlp.normwise_rel_err(to_np(g), r) for n, g, r in
            (("out", out, fw.out), ("dx", dx, bw.dx), ("dprob", dprob, bw.dprob), ("dw1", dw1, bw.dw1), ("dw2", dw2, bw.dw2))}
    log(" ".join(f"{k}={v:.2e}" for k, v in errs.items()))
    assert all(v < MXFP8_TOL for v in errs.values()), errs
    if case[6]:
        for e, n in enumerate(case[6]):
            if n == 0:
                assert not dw1[e].any() and not dw2[e].any()
    # the same call without saving, and with cached weights, gives the same bits
    plain, _ = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, "fp8_block")
    wq = m.quantize_weights(d.w1, d.w2, "fp8_block")
    cached, _ = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, "fp8_block", w_quant=wq)
    wt = m.quantize_weights(d.w1, d.w2, "fp8_block", transposed=True)
    again = m.moe_grouped_mlp_bwd(d.dy, ctx, d.w1, d.w2, dw_dtype=dw, w_quant_t=wt)
    torch.cuda.synchronize()
    assert torch.equal(out, plain) and torch.equal(out, cached)
    assert all(torch.equal(x, y) for x, y in zip((dx, dprob, dw1, dw2), again))


@gpu
def test_expert_lists_and_h_f32():
    """Weights as a list of tensors, and the fp32 h ahead of its quantization."""
    m = need_gpu()
    cfg, inp = _inputs(CASES[1])
    d = inp.to("cuda")
    out, ctx = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, [w.clone() for w in d.w1], [w.clone() for w in d.w2],
                                     "fp8_block", debug_h=True)
    ref, _ = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, "fp8_block")
    fw, _ = _oracle(cfg, inp)
    assert torch.equal(out, ref)
    assert mlp.normwise_rel_err(to_np(ctx["debug"]["h_f32"]), fw.h) < MXFP8_TOL


@gpu
def test_dropped_pairs_and_refusals():
    m = need_gpu()
    cfg, inp = _inputs(CASES[1])
    d = inp.to("cuda")
    bad = d.topk_idx.clone()
    bad[5, 1] = 99
    bad[6, 0] = -3
    out, ctx = m.moe_grouped_mlp_fwd(d.x, bad, d.topk_prob, d.w1, d.w2, "fp8_block", save_for_backward=True)
    dx, dprob, dw1, dw2 = m.moe_grouped_mlp_bwd(d.dy, ctx, d.w1, d.w2)
    good, _ = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, "fp8_block")
    torch.cuda.synchronize()
    assert m.moe_read_device_error(ctx["error_flag"]) == 1
    ok = torch.ones(cfg.T, dtype=torch.bool, device="cuda")
    ok[[5, 6]] = False
    # (rows move within their expert's tiles: sums of the same products, in the same order)
    assert torch.equal(out[ok], good[ok])
    assert all(torch.isfinite(t.float()).all() for t in (out, dx, dw1, dw2))
    with pytest.raises(m.MoeError):
        m.moe_grouped_mlp_fwd_loop(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, [128, 0, 0, 0], "fp8_block")
    with pytest.raises(m.MoeError):
        m.moe_grouped_mlp_fwd(d.x[:, :192].contiguous(), d.topk_idx, d.topk_prob, d.w1[:, :, :192].contiguous(),
                              d.w2[:, :192].contiguous(), "fp8_block")


def _step(m, x, lg, mask, w1, w2, dy, dl, k):
    idx, prob, counts, losses = m.moe_route_balance(lg, k, token_mask=mask)
    out, ctx = m.moe_grouped_mlp_fwd(x, idx, prob, w1, w2, "fp8_block", save_for_backward=True)
    dx, dprob, dw1, dw2 = m.moe_grouped_mlp_bwd(dy, ctx, w1, w2)
    dlg = m.moe_route_balance_bwd(lg, idx, prob, counts, dprob, dl, token_mask=mask)
    return out, losses, dx, dw1, dw2, dlg


@gpu
def test_router_and_experts_together():
    """A layer's training step: route, expert MLP, backward, and the gradient of the logits from the
    experts' dprob and both losses -- against the oracle, in a captured graph, and on another stream."""
    m = need_gpu()
    T, H, I, E, k = 384, 256, 256, 8, 2
    cfg = cfg_small(T=T, H=H, I=I, E=E, k=k, seed=77)
    inp = make_inputs(cfg, with_dy=True)
    d = inp.to("cuda")
    lg = torch.from_numpy(np.random.default_rng(4).standard_normal((T, E)).astype(np.float32))
    mask = torch.ones(T, dtype=torch.bool)
    mask[350:] = False
    inp.dy[350:] = 0                      # padding tokens have no gradient of their own
    dy = inp.dy.cuda()
    dl = torch.tensor([0.02, 0.001])
    args = (m, d.x, lg.cuda(), mask.cuda(), d.w1, d.w2, dy, dl.cuda(), k)
    out, losses, dx, dw1, dw2, dlg = want = _step(*args)
    torch.cuda.synchronize()
    idx, prob, counts, rl = balance.forward(lg, k, mask.numpy())
    p32 = torch.from_numpy(prob.astype(np.float32))
    fw = mlp.forward(inp.x, idx, p32, inp.w1, inp.w2, "fp8_block", "bf16")
    bw = mlp.backward(fw, inp.x, inp.dy, inp.w1, inp.w2)
    rd, _ = balance.backward(lg, idx, prob, counts, bw.dprob, dl.double().numpy(), mask.numpy())
    errs = {n: mlp.normwise_rel_err(to_np(g), r) for n, g, r in
            (("out", out, fw.out), ("dx", dx, bw.dx), ("dw1", dw1, bw.dw1), ("dw2", dw2, bw.dw2), ("dlogits", dlg, rd))}
    log(" ".join(f"{k}={v:.2e}" for k, v in errs.items()))
    assert all(v < MXFP8_TOL for v in errs.values()), errs
    assert np.abs(losses.cpu().double().numpy() - rl).max() <= 80 * 2.0 ** -24 * np.abs(rl).max()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = _step(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    ws = [torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, prob, counts, l2 = m.moe_route_balance(args[2], k, token_mask=args[3])
        o2, ctx = m.moe_grouped_mlp_fwd(d.x, idx, prob, d.w1, d.w2, "fp8_block", save_for_backward=True, workspace=ws[0])
        dx2, dp2, a2, b2 = m.moe_grouped_mlp_bwd(dy, ctx, d.w1, d.w2, workspace=ws[1])
        c2 = m.moe_route_balance_bwd(args[2], idx, prob, counts, dp2, args[7], token_mask=args[3])
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        _step(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((o2, l2, dx2, a2, b2, c2), want))


@gpu
@pytest.mark.parametrize("dw", [torch.float32, torch.bfloat16], ids=["dw-f32", "dw-bf16"])
def test_weight_gradients_split_along_the_tokens(dw):
    """Few, long tiles: the layer's weight gradients are split into parts and joined through its table of
    outputs and its own scratch, to the bits of the operators called one by one."""
    m = need_gpu()
    case = (6000, 128, 128, 2, 1, "bf16", [5900, 100])
    cfg, inp = _inputs(case)
    log(f"fp8_block mlp {case} {dw}")
    d = inp.to("cuda")
    w1, w2 = [w.clone() for w in d.w1], [w.clone() for w in d.w2]
    out, ctx = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, w1, w2, "fp8_block", save_for_backward=True)
    dx, dprob, dw1, dw2 = m.moe_grouped_mlp_bwd(d.dy, ctx, w1, w2, dw_dtype=dw)
    off = ctx["perm"]["offsets"]
    dz = d.dy[ctx["perm"]["src_index"].long()].contiguous()
    dzt = m.fp8_block_quantize(dz, axis=1, group_offsets=off)
    ht = m.fp8_block_quantize(ctx["saved"]["h"], axis=1, group_offsets=off)
    alone = m.fp8_block_grouped_wgrad(*dzt, *ht, off, out_dtype=dw)
    torch.cuda.synchronize()
    fw, bw = _oracle(cfg, inp)
    errs = {n: mlp.normwise_rel_err(to_np(g), r) for n, g, r in
            (("out", out, fw.out), ("dx", dx, bw.dx), ("dprob", dprob, bw.dprob), ("dw1", dw1, bw.dw1), ("dw2", dw2, bw.dw2))}
    log(" ".join(f"{k}={v:.2e}" for k, v in errs.items()))
    assert all(v < MXFP8_TOL for v in errs.values()), errs
    assert torch.equal(dw2, alone)


@gpu
@pytest.mark.parametrize("compute", ["bf16", "mxfp8", "fp8_block"])
def test_graphs_of_two_layers_replayed_at_once(compute):
    """Forward and backward of two layers, each captured with the workspaces that the calls take by themselves, on two
    streams."""
    m = need_gpu()
    log(f"two graphs {compute}")
    steps = []
    for case in ((300, 256, 384, 4, 2, "bf16", None), (257, 384, 256, 5, 1, "bf16", None)):
        cfg, inp = _inputs(case)
        d = inp.to("cuda")

        def step(d=d):
            out, ctx = m.moe_grouped_mlp_fwd(d.x, d.topk_idx, d.topk_prob, d.w1, d.w2, compute, save_for_backward=True)
            return (out, *m.moe_grouped_mlp_bwd(d.dy, ctx, d.w1, d.w2))
        steps.append(step)
    want = [s() for s in steps]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(s())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        steps[0]()
        torch.cuda.synchronize()

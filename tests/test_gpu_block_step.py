"""One training step of a mixture-of-experts block through the operators in their order of use: norm -> router -> layer
and a shared expert's product on the norm's codes -> gradients of all of them -> clipping; against fp64 autograd.

Tolerance: bf16 activations are rounded about ten times on the way (half steps 2^-9 each, independent: 10^0.5 2^-9 =
0.6 %), the shared expert's operands once each to E4M3 (half steps 2^-4 at most, 2.6 % in the mean square, on a quarter
of the output): 2e-2 normwise, 5e-2 for what passes the E4M3 product.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, log, need_gpu

B = torch.bfloat16
T, H, I, E, K = 300, 256, 128, 16, 4
ROUTE = dict(score="sigmoid", renormalize=True, scale=2.5)


def _state():
    g = torch.Generator().manual_seed(11)
    r = lambda *s, k=1.0: torch.randn(s, generator=g) * k
    return {"x": r(T, H).to(B), "res": r(T, H).to(B), "wn": (1 + 0.1 * r(H)).to(B), "wr": r(H, E, k=H ** -0.5).to(B),
            "w1": r(E, 2 * I, H, k=H ** -0.5).to(B), "w2": r(E, H, I, k=I ** -0.5).to(B), "ws": r(H, H, k=H ** -0.5).to(B),
            "bias": r(E, k=0.1), "dout": r(T, H).to(B)}


def _step(m, s, offsets, ws, wst):
    y, total, codes, scales = m.moe_add_rmsnorm(s["x"], s["wn"], residual=s["res"], codes=True)
    logits = (y @ s["wr"]).float()
    idx, prob, counts = m.moe_route_grouped(logits, K, bias=s["bias"], groups=4, topk_groups=2, count=True, **ROUTE)
    out, ctx = m.moe_grouped_mlp_fwd(y, idx, prob, s["w1"], s["w2"], "bf16", save_for_backward=True)
    shared = m.fp8_block_grouped_gemm(codes, scales, *ws, offsets)
    # backward of total + out + shared
    dy, dprob, dw1, dw2 = m.moe_grouped_mlp_bwd(s["dout"], ctx, s["w1"], s["w2"])
    dcodes, dscales = m.fp8_block_quantize(s["dout"])
    dy = dy + m.fp8_block_grouped_gemm(dcodes, dscales, *wst, offsets)
    dlogits = m.moe_route_grouped_bwd(logits, idx, prob, dprob, **ROUTE)
    dwr = (y.float().t().contiguous() @ dlogits)
    dy = dy + (dlogits @ s["wr"].float().t().contiguous()).to(B)
    dx, dwn = m.moe_add_rmsnorm_bwd(dy, total, s["wn"], ds=s["dout"])
    grads = [dw1, dw2, dwr, dwn]
    raw = [t.clone() for t in grads]
    norm = m.moe_grad_clip(grads, 1.0)
    return {"out": total.float() + out.float() + shared.float(), "idx": idx, "counts": counts, "prob": prob, "dx": dx,
            "norm": norm, "raw": raw, "grads": grads, "logits": logits,
            "split_sizes": ctx["perm"]["split_sizes"]}


def _reference(s, idx):
    d = {k: v.double().requires_grad_(k not in ("bias", "dout")) for k, v in s.items()}
    total = (d["x"] + d["res"])
    y = total * torch.rsqrt(total.square().mean(1, keepdim=True) + 1e-6) * d["wn"]
    sc = torch.sigmoid(y @ d["wr"]).gather(1, idx.long())
    prob = 2.5 * sc / sc.sum(1, keepdim=True)
    out = total + y @ d["ws"].t()
    for j in range(K):
        gu = torch.stack([d["w1"][e] @ y[t] for t, e in enumerate(idx[:, j].tolist())])
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:] * prob[:, j:j + 1]
        out = out + torch.stack([d["w2"][e] @ h[t] for t, e in enumerate(idx[:, j].tolist())])
    (out * d["dout"]).sum().backward()
    return out.detach(), prob.detach(), d


def _err(a, b):
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    return float((a - b).norm() / b.norm())


@gpu
def test_training_step_of_a_block_eager_and_captured():
    m = need_gpu()
    cpu = _state()
    s = {k: v.cuda() for k, v in cpu.items()}
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ws = m.fp8_block_quantize_weights(s["ws"][None])
    wst = m.fp8_block_quantize_weights(s["ws"][None], transposed=True)
    got = _step(m, s, offsets, ws, wst)
    torch.cuda.synchronize()
    assert torch.equal(got["counts"], got["split_sizes"])           # what the layer's permutation counts
    out, prob, d = _reference(cpu, got["idx"].cpu())
    for name, a, b, tol in (("out", got["out"], out, 5e-2), ("prob", got["prob"], prob, 2e-2), ("dx", got["dx"], d["x"].grad, 5e-2),
                            ("dw1", got["raw"][0], d["w1"].grad, 2e-2), ("dw2", got["raw"][1], d["w2"].grad, 2e-2),
                            ("dwr", got["raw"][2], d["wr"].grad, 2e-2), ("dwn", got["raw"][3], d["wn"].grad, 5e-2)):
        e = _err(a, b)
        log(f"{name}: {e:.2e}")
        assert e < tol, name
    total = float(np.sqrt(sum(float(t.double().square().sum()) for t in got["raw"])))
    assert abs(float(got["norm"]) - total) <= 1e-6 * total
    assert abs(float(np.sqrt(sum(float(t.double().square().sum()) for t in got["grads"]))) - 1.0) <= 1e-5
    # the routing is the oracle's for the same logits
    from oracle import group_route
    ri, _, _ = group_route.forward(got["logits"].cpu(), K, cpu["bias"], "sigmoid", 4, 2, 2)
    np.testing.assert_array_equal(got["idx"].cpu().numpy(), ri)
    # captured, and replayed with eager work between
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(m, s, offsets, ws, wst)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = _step(m, s, offsets, ws, wst)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "idx", "counts", "prob", "dx", "norm"):
            assert torch.equal(cap[name], got[name]), name
        assert all(torch.equal(a, b) for a, b in zip(cap["grads"], got["grads"]))
        _step(m, s, offsets, ws, wst)
        torch.cuda.synchronize()

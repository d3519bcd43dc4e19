"""The operators around a mixture-of-experts layer in a training or serving step, as measured cases.

  route_fwd   routing by sigmoid or softmax scores: a bias that counts in the selection alone, expert groups of
              which a token keeps the best, top-k, weights renormalised and scaled; per-expert counts
  route_bwd   the gradient of the routing weights with respect to the logits
  norm_fwd    residual addition and root-mean-square norm ahead of the layer, its output in the activations'
              type, in E4M3 with one fp32 scale per 128 columns (a block-scaled product's operand), or both
  norm_bwd    the norm's gradients, with the residual stream's own added
  clip        the global norm of many gradients, and their clipped copies
  clip_shared the gradients clipped in place by a norm that is known already (summed over all ranks)

Sizes are those of moe_inputs/configs.py (the Mixtral layer: H 4096, 8 experts; the fine-grained one: H 2048,
I 1408, 64 experts) and of the limits that include/moe.h sets (256 experts), and odd ones between.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126          # the smallest normal fp32: scales never go below it
F8 = torch.float8_e4m3fn
EPS = 1e-6                  # of the norm, and beside the gradients' norm


def listed():
    return [
        # decoding one token at the largest expert count, half of 8 groups kept: all latency
        dict(name="route_fwd_t1_e256_g8", op="route_fwd", T=1, E=256, k=8, dtype="f32", score="sigmoid", bias=True, G=8,
             kg=4, best=2, renorm=True, scale=2.5, counts=False, masked=False),
        # a training batch with padding, the counts taken for the bias's next update
        dict(name="route_fwd_t131072_e256_g8", op="route_fwd", T=131072, E=256, k=8, dtype="f32", score="sigmoid",
             bias=True, G=8, kg=4, best=2, renorm=True, scale=2.5, counts=True, masked=True),
        # softmax scores, groups by their best expert, weights left as they are; odd sizes
        dict(name="route_fwd_t50021_e160_g8", op="route_fwd", T=50021, E=160, k=6, dtype="bf16", score="softmax",
             bias=False, G=8, kg=3, best=1, renorm=False, scale=16.0, counts=False, masked=False),
        # the backward of such training batches, k selected logits a token
        dict(name="route_bwd_t131072_e256", op="route_bwd", T=131072, E=256, k=8, dtype="f32", score="sigmoid",
             renorm=True, scale=2.5),
        # softmax weights that are not renormalised: every logit has a gradient
        dict(name="route_bwd_t30011_e157", op="route_bwd", T=30011, E=157, k=7, dtype="bf16", score="softmax",
             renorm=False, scale=1.0),
        # decoding one token of the Mixtral layer
        dict(name="norm_fwd_t1_h4096", op="norm_fwd", T=1, H=4096, dtype="bf16", wdtype="bf16", residual=True, to="both"),
        # 16384 tokens ahead of the router (bf16) and a shared expert's product (codes)
        dict(name="norm_fwd_t16384_h4096", op="norm_fwd", T=16384, H=4096, dtype="bf16", wdtype="bf16", residual=True,
             to="both"),
        # an odd width in fp32: rows that start at any 4-byte address
        dict(name="norm_fwd_t100003_h1003", op="norm_fwd", T=100003, H=1003, dtype="f32", wdtype="f32", residual=False,
             to="y"),
        # the Mixtral layer's width in training, the residual stream's gradient added
        dict(name="norm_bwd_t16384_h4096", op="norm_bwd", T=16384, H=4096, dtype="bf16", wdtype="bf16", ds=True),
        # an odd width in fp32, no residual
        dict(name="norm_bwd_t20011_h1407", op="norm_bwd", T=20011, H=1407, dtype="f32", wdtype="f32", ds=False),
        # the fine-grained layer's weight gradients in fp32, clipped into a bf16 bucket
        dict(name="clip_e64", op="clip", n=2, lo=64 * 2048 * 1408, hi=64 * 2816 * 2048, kinds="f32", out="bf16", sizes=0),
        # what else a model has: many tensors from one value up, of both types
        dict(name="clip_ragged_200", op="clip", n=200, lo=1, hi=3000000, kinds="both", out="f32", sizes=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route_fwd", "route_fwd", "route_bwd", "norm_fwd", "norm_fwd", "norm_bwd", "clip", "clip_shared"])
    dtype = rng.choice(["f32", "bf16"])
    score = rng.choice(["sigmoid", "softmax"])
    renorm, scale = rng.random() < 0.6, rng.choice([1.0, 2.5, 16.0])
    if op == "route_fwd":
        G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        n = _log(rng, 2, 256 // G)
        kg = rng.randint(1, G)
        return dict(op=op, T=_log(rng, 1, 131072), E=G * n, k=rng.randint(1, min(kg * n, 16)), dtype=dtype, score=score,
                    bias=rng.random() < 0.6, G=G, kg=kg, best=rng.randint(1, 2), renorm=renorm, scale=scale,
                    counts=rng.random() < 0.5, masked=rng.random() < 0.5)
    if op == "route_bwd":
        E = _log(rng, 2, 256)
        return dict(op=op, T=_log(rng, 1, 131072), E=E, k=rng.randint(1, min(E, 16)), dtype=dtype, score=score,
                    renorm=renorm, scale=scale)
    if op in ("norm_fwd", "norm_bwd"):
        aligned = rng.random() < 0.5
        while True:
            H = 128 * _log(rng, 1, 128) if aligned else _log(rng, 2, 16384)
            case = dict(op=op, T=_log(rng, 1, 131072), H=H, dtype=dtype, wdtype=rng.choice([dtype, "f32"]))
            if op == "norm_fwd":
                case.update(residual=rng.random() < 0.6, to=rng.choice(["y", "codes", "both"]) if aligned else "y")
            else:
                case.update(ds=rng.random() < 0.6)
            if work(case)["bytes"] <= (8.0e8 if op == "norm_fwd" else 5.3e8):
                return case
    while True:
        n = _log(rng, 1, 300)
        lo = _log(rng, 1, 4096)
        case = dict(op=op, n=n, lo=lo, hi=lo * _log(rng, 1, 100000), kinds=rng.choice(["f32", "bf16", "both"]),
                    out=rng.choice(["f32", "bf16"]), sizes=rng.randint(2, 1 << 20))
        if work(case)["bytes"] <= 3.3e9:
            return case


def _torch_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _bytes(name):
    return 4 if name == "f32" else 2


def _tensors(case):
    """(values, type) of each gradient: spread over lo .. hi by their logarithm, from the case alone."""
    rng, n = random.Random(case["sizes"]), case["n"]
    if n == 2 and case["sizes"] == 0:          # the listed layer: its two tables
        return [(case["hi"], "f32"), (case["lo"], "f32")]
    kinds = ["f32", "bf16"] if case["kinds"] == "both" else [case["kinds"]]
    return [(_log(rng, case["lo"], case["hi"]), rng.choice(kinds)) for _ in range(n)]


def work(case):
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        row = T * E * _bytes(case["dtype"])
        if op == "route_fwd":
            more = (4 * E if case["bias"] else 0) + (4 * E if case["counts"] else 0)
            more += T if case["masked"] and case["counts"] else 0
            return {"bytes": row + 8 * T * k + more, "flops": 12 * T * E}
        dense = case["score"] == "softmax" and not case["renorm"]
        read = row if dense else T * k * _bytes(case["dtype"]) if case["score"] == "sigmoid" else 0
        return {"bytes": row + read + 12 * T * k, "flops": (6 * T * E if dense else 0) + 12 * T * k}
    if op in ("norm_fwd", "norm_bwd"):
        T, H, b = case["T"], case["H"], _bytes(case["dtype"])
        w = H * _bytes(case["wdtype"])
        if op == "norm_fwd":
            n = b * (3 if case["residual"] else 1) + (b if case["to"] != "codes" else 0)
            n = T * H * n + (T * H + T * H // 32 if case["to"] != "y" else 0)
            return {"bytes": n + w, "flops": 8 * T * H}
        return {"bytes": T * H * b * (4 if case["ds"] else 3) + w + 4 * H, "flops": 14 * T * H}
    sizes = _tensors(case)
    total = sum(n for n, _ in sizes)
    read = sum(n * _bytes(d) for n, d in sizes)
    if op == "clip":
        return {"bytes": read + total * _bytes(case["out"]), "flops": 3 * total}
    return {"bytes": 2 * read, "flops": total}


# ---------------------------------------------------------------------------- inputs

def _activations(gen, rows, cols, dtype):
    """Token rows as a layer sees them: unit normal, a few channels far larger than the rest."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.exp(torch.randn((1, cols), generator=gen, device="cuda").clamp_(-2, 2).mul_(0.7))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op in ("route_fwd", "route_bwd"):
        T, E = case["T"], case["E"]
        s["logits"] = (torch.randn((T, E), generator=gen, device="cuda") * 1.5).to(_torch_dtype(case["dtype"]))
        if op == "route_fwd":
            s["b"] = s["mask"] = None
            if case["bias"]:       # moved up or down by small steps in training, for balance
                step = 0.1 if case["score"] == "sigmoid" else 0.3 / E
                s["b"] = torch.randn(E, generator=gen, device="cuda") * step
            if case["masked"]:     # sequences end in padding tokens, which do not count
                s["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.85
            return s
        s["idx"], s["prob"], _ = _route(s["logits"], None, None, dict(case, G=1, counts=False))
        s["dprob"] = torch.randn((T, case["k"]), generator=gen, device="cuda") / T
        return s
    if op in ("norm_fwd", "norm_bwd"):
        T, H, dt = case["T"], case["H"], _torch_dtype(case["dtype"])
        s["w"] = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(_torch_dtype(case["wdtype"]))
        s["x"] = _activations(gen, T, H, dt)
        if op == "norm_fwd":
            s["r"] = _activations(gen, T, H, dt) if case["residual"] else None
        else:
            s["dy"] = (torch.randn((T, H), generator=gen, device="cuda") * 0.01).to(dt)
            s["dsum"] = (torch.randn((T, H), generator=gen, device="cuda") * 0.01).to(dt) if case["ds"] else None
        return s
    # gradients in buckets, one of each type, as a data-parallel program keeps them
    sizes = _tensors(case)
    buckets = {}
    for kind in ("f32", "bf16"):
        total = sum(n for n, d in sizes if d == kind)
        buckets[kind] = torch.empty(total, device="cuda", dtype=_torch_dtype(kind))
        for at in range(0, total, 1 << 27):
            part = buckets[kind][at:at + (1 << 27)]
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * 0.01)
    total = sum(n for n, _ in sizes)
    s["buckets"] = buckets
    s["grads"] = _views(buckets, sizes)
    if op == "clip":
        s["bucket"] = torch.empty(total, device="cuda", dtype=_torch_dtype(case["out"]))
        s["out"] = list(s["bucket"].split([n for n, _ in sizes]))
        s["max_norm"] = 0.3 * 0.01 * math.sqrt(total)
    else:
        # the other ranks' gradients are as large: 8 ranks, a norm 2 % over the limit
        s["sumsq"] = (8.0 + torch.rand(1, generator=gen, device="cuda", dtype=torch.float64)) * (1e-4 * total)
        s["max_norm"] = 0.98 * 0.01 * math.sqrt(8.5 * total)
    s["table"] = None
    if own:     # the plan that a training program keeps beside its buckets
        import mixture_experts_grouped_permute_amd as m
        s["table"] = m.GradTable(s["grads"], s["out"] if op == "clip" else None)
    return s


def _views(buckets, sizes):
    at, out = {"f32": 0, "bf16": 0}, []
    for n, d in sizes:
        out.append(buckets[d][at[d]:at[d] + n])
        at[d] += n
    return out


# ---------------------------------------------------------------------------- plain forms

def _scores(l, score):
    """Scores in 64 bits; a row without a logit above -inf has zeros."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    return torch.where(total == 0, 0.0, e / total)


def _route(logits, bias, mask, c):
    """ids, weights and counts.  Scores in 64 bits: the order of two that are nearly equal hangs on their last bits."""
    T, E = logits.shape
    k, G = c["k"], c["G"]
    l = logits.double()
    s = _scores(l, c["score"])
    v = s if bias is None else s + bias.double()
    v = torch.where(l == -math.inf, -math.inf, v)
    if G > 1:
        v = v.view(T, G, E // G)
        best = torch.sort(v, dim=2, descending=True, stable=True).values[:, :, :c["best"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kg"]]
        stays = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        v = torch.where(stays[:, :, None], v, -math.inf).view(T, E)
    v, idx = torch.sort(v, dim=1, descending=True, stable=True)     # equal: the lower id first
    v, idx = v[:, :k], idx[:, :k]
    w = torch.where(v == -math.inf, 0.0, torch.gather(s, 1, idx))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    w = (w * c["scale"]).float()
    counts = None
    if c["counts"]:
        live = idx if mask is None else torch.where(mask[:, None], idx, E)
        counts = torch.bincount(live.reshape(-1), minlength=E + 1)[:E].to(torch.int32)
    return idx.to(torch.int32), w, counts


def _route_bwd(logits, idx, prob, dprob, c):
    l, i = logits.double(), idx.long()
    w, g = prob.double(), dprob.double()
    if c["renorm"]:
        g = g - (w * g).sum(1, keepdim=True) / c["scale"]
    d = w * g
    if c["score"] == "sigmoid":
        d = d / (1 + torch.exp(torch.gather(l, 1, i)))      # 1 - sigmoid
    out = torch.zeros_like(l).scatter_add_(1, i, d)
    if c["score"] == "softmax" and not c["renorm"]:
        out -= _scores(l, "softmax") * d.sum(1, keepdim=True)
    return out.to(logits.dtype)


def _quant_rows(v):
    """codes [T, H] and scales [H / 128, T] of fp32 values."""
    T, H = v.shape
    v = v.view(T, H // 128, 128)
    amax = v.abs().amax(2)
    none = amax == 0
    factor = torch.where(none, 1.0, (E4M3_MAX / amax).clamp(max=1 / TINY))
    scale = torch.where(none, 1.0, (amax / E4M3_MAX).clamp(min=TINY))
    return (v * factor[:, :, None]).to(F8).view(T, H), scale.t().contiguous()


def _norm(s):
    x = s["x"].float()
    out = {}
    if s["r"] is not None:
        out["s"] = (x + s["r"].float()).to(s["x"].dtype)    # the sum as the next layer reads it: the norm is its
        x = out["s"].float()
    y = x * (1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)) * s["w"].float()
    if s["to"] != "codes":
        out["y"] = y.to(s["x"].dtype)
    if s["to"] != "y":
        out["codes"], out["scales"] = _quant_rows(y)
    return out


def _norm_bwd(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    x = x * rstd
    g = dy * w
    dx = rstd * (g - x * (g * x).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * x).sum(0, dtype=torch.float64).float()}


def _sumsq(grads):
    parts = [sum((p.float() * p.float()).sum(dtype=torch.float64) for p in g.split(1 << 27)) for g in grads]
    return torch.stack(parts).sum()


def _clip_to(grads, out, sumsq, max_norm):
    norm = torch.sqrt(sumsq)
    c = (max_norm / (norm + EPS)).clamp(max=1.0).float()
    for g, o in zip(grads, out):
        for a, b in zip(g.split(1 << 27), o.split(1 << 27)):
            b.copy_(a.float() * c)
    return norm.float().reshape(1)


def run(s):
    op = s["op"]
    if own:
        import mixture_experts_grouped_permute_amd as m
        if op == "route_fwd":
            idx, prob, counts = m.moe_route_grouped(
                s["logits"], s["k"], bias=s["b"], score=s["score"], groups=s["G"], topk_groups=s["kg"],
                group_best=s["best"], renormalize=s["renorm"], scale=s["scale"], token_mask=s["mask"] if s["counts"] else None,
                count=s["counts"])
            return {"idx": idx, "prob": prob, "counts": counts}
        if op == "route_bwd":
            return m.moe_route_grouped_bwd(s["logits"], s["idx"], s["prob"], s["dprob"], score=s["score"],
                                           renormalize=s["renorm"], scale=s["scale"])
        if op == "norm_fwd":
            y, total, codes, scales = m.moe_add_rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS, y=s["to"] != "codes",
                                                        codes=s["to"] != "y")
            out = {"s": total} if s["r"] is not None else {}
            out.update({"y": y} if y is not None else {})
            out.update({"codes": codes.view(F8), "scales": scales} if codes is not None else {})
            return out
        if op == "norm_bwd":
            dx, dw = m.moe_add_rmsnorm_bwd(s["dy"], s["x"], s["w"], ds=s["dsum"], eps=EPS)
            return {"dx": dx, "dw": dw}
        if op == "clip":
            return {"norm": m.moe_grad_clip(s["table"], s["max_norm"]), "out": s["bucket"]}
        return {"norm": m.moe_grad_clip(s["table"], s["max_norm"], sumsq=s["sumsq"]), **_held(s["buckets"])}
    if op == "route_fwd":
        idx, prob, counts = _route(s["logits"], s["b"], s["mask"], s)
        return {"idx": idx, "prob": prob, "counts": counts}
    if op == "route_bwd":
        return _route_bwd(s["logits"], s["idx"], s["prob"], s["dprob"], s)
    if op == "norm_fwd":
        return _norm(s)
    if op == "norm_bwd":
        return _norm_bwd(s)
    if op == "clip":
        return {"norm": _clip_to(s["grads"], s["out"], _sumsq(s["grads"]), s["max_norm"]), "out": s["bucket"]}
    return {"norm": _clip_to(s["grads"], s["grads"], s["sumsq"], s["max_norm"]), **_held(s["buckets"])}


def _held(buckets):
    return {kind: b for kind, b in buckets.items() if b.numel()}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definitions, in 64 bits; whole numbers and codes (whose rounding borders move with the last bit of a
    factor) have no such value."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "route_fwd":
        l = s["logits"].to(torch.float64)
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        c = score if s["b"] is None else score + s["b"]
        if case["G"] > 1:
            per = torch.stack([t.topk(case["best"], 1).values.sum(1) for t in c.chunk(case["G"], 1)], 1)
            rank = torch.argsort(torch.argsort(per, dim=1, descending=True, stable=True), dim=1)
            c = c.masked_fill((rank >= case["kg"]).repeat_interleave(case["E"] // case["G"], 1), -1e9)
        w = score.gather(1, torch.argsort(c, dim=1, descending=True, stable=True)[:, :case["k"]])
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"idx": None, "prob": w * case["scale"], "counts": None}
    if op == "route_bwd":
        # through the Jacobian of the scores, selected columns first
        l, ids = s["logits"].to(torch.float64), s["idx"].to(torch.int64)
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        p = score.gather(1, ids)
        g = s["dprob"].to(torch.float64) * case["scale"]
        if case["renorm"]:
            total = p.sum(1, keepdim=True)
            g = (g - (g * p).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(l).scatter_(1, ids, g)
        if case["score"] == "sigmoid":
            return ds * score * (1 - score)
        return score * (ds - (ds * score).sum(1, keepdim=True))
    if op == "norm_fwd":
        out = {}
        v = s["x"].to(torch.float64)
        if s["r"] is not None:
            v = (v + s["r"]).to(s["x"].dtype).to(torch.float64)
            out["s"] = v
        y = v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["w"]
        if case["to"] != "codes":
            out["y"] = y
        if case["to"] != "y":
            amax = y.abs().reshape(case["T"], -1, 128).amax(2).t()
            out["codes"], out["scales"] = None, torch.where(amax > 0, amax / 448, 1.0)
        return out
    if op == "norm_bwd":
        v, dy, w = (s[n].to(torch.float64) for n in ("x", "dy", "w"))
        H = case["H"]
        ms = v.pow(2).mean(1, keepdim=True) + EPS
        dx = dy * w / ms.sqrt() - v * ((dy * w * v).sum(1, keepdim=True) / (H * ms.pow(1.5)))
        if s["dsum"] is not None:
            dx = dx + s["dsum"]
        return {"dx": dx, "dw": (dy * v / ms.sqrt()).sum(0)}
    if op == "clip":
        total = sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"])
    else:
        total = float(s["sumsq"])
    norm = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (norm + EPS))
    norm = torch.tensor([norm], dtype=torch.float64)
    if op == "clip":
        return {"norm": norm, "out": torch.cat([g.to(torch.float64) * c for g in s["grads"]])}
    return {"norm": norm, **{kind: b.to(torch.float64) * c for kind, b in _held(s["buckets"]).items()}}

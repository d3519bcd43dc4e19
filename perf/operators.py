"""The operators of the training router and of block-scaled FP8 expert products, as measured cases.

Two families, which a mixture-of-experts layer uses one after the other:

  route_fwd    top-k routing with per-expert counts, the load-balance loss and the router z-loss
  route_bwd    the gradient of the routing weights and of both losses with respect to the logits
  quant_rows   E4M3 codes with one fp32 scale per row and 128 columns (a product's activations)
  quant_cols   the same along tokens, 128 tokens of one expert to a block, transposed (a weight
               gradient's operands)
  quant_weights  E4M3 codes with one fp32 scale per 128 x 128 block of every expert's matrix
  gemm         the grouped product of such activations and weights (forward, and dgrad with the
               transposed weights)
  wgrad        the grouped weight gradient of two token-axis operands

Sizes are those of moe_inputs/configs.py (the Mixtral layer: H 4096, I 14336, 8 experts, top-2; the
fine-grained one: H 2048, I 1408, 64 experts, top-8; the tiny one: 256 tokens, 4 experts, top-2) and
of the limits that include/moe.h sets (256 experts).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126          # the smallest normal fp32: scales never go below it
F8 = torch.float8_e4m3fn


def listed():
    return [
        # the tiny layer's router: all latency
        dict(name="route_fwd_t256_e4", op="route_fwd", T=256, E=4, k=2, dtype="f32", masked=False),
        # a padded batch of a fine-grained model at the largest expert count
        dict(name="route_fwd_t131072_e256", op="route_fwd", T=131072, E=256, k=8, dtype="f32", masked=True),
        # the fine-grained layer's router in training, logits in bf16
        dict(name="route_bwd_t16384_e64", op="route_bwd", T=16384, E=64, k=8, dtype="bf16", masked=False),
        # odd sizes: tokens, experts and k that divide nothing, with padding tokens
        dict(name="route_bwd_t100003_e157", op="route_bwd", T=100003, E=157, k=7, dtype="f32", masked=True),
        # permuted activations of the Mixtral layer (8192 tokens, top-2) ahead of its gate-up product
        dict(name="quant_rows_16384x4096", op="quant_rows", R=16384, C=4096, dtype="bf16"),
        # the fine-grained layer's h along tokens, ahead of its down projection's weight gradient
        dict(name="quant_cols_131072x1408_e64", op="quant_cols", R=131072, C=1408, E=64, skew=1.0, dtype="bf16"),
        # the Mixtral layer's down weights for dgrad: the transposed codes
        dict(name="quant_weights_t_e8", op="quant_weights", E=8, N=4096, K=14336, transposed=True),
        # decoding: a batch of 4 tokens, top-2, through the Mixtral layer's gate-up weights
        dict(name="gemm_decode_r8_e8", op="gemm", R=8, E=8, N=28672, K=4096, skew=0.0, out="bf16"),
        # the fine-grained layer's gate-up product, tokens skewed over the experts
        dict(name="gemm_r131072_e64", op="gemm", R=131072, E=64, N=2816, K=2048, skew=1.0, out="bf16"),
        # the Mixtral layer's down projection, 8192 tokens
        dict(name="gemm_r16384_e8", op="gemm", R=16384, E=8, N=4096, K=14336, skew=1.2, out="bf16"),
        # weight gradients of the fine-grained layer's gate-up and the Mixtral layer's down projection
        dict(name="wgrad_r131072_e64", op="wgrad", R=131072, E=64, N=2816, K=2048, skew=1.0, out="f32"),
        dict(name="wgrad_r16384_e8", op="wgrad", R=16384, E=8, N=4096, K=14336, skew=1.2, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _fits(case):
    """No dearer than the largest listed cases: 1.93e12 operations (gemm, wgrad), 1.4 GB moved (the others)."""
    w = work(case)
    return w["flops"] <= 1.95e12 if case["op"] in ("gemm", "wgrad") else w["bytes"] <= 1.4e9


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "quant_rows", "quant_cols", "quant_weights", "gemm", "gemm", "wgrad"])
    while True:
        if op in ("route_fwd", "route_bwd"):
            E = _log(rng, 2, 256)
            case = dict(op=op, T=_log(rng, 1, 131072), E=E, k=rng.randint(1, min(E, 16)),
                        dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
        elif op == "quant_rows":
            case = dict(op=op, R=_log(rng, 1, 131072), C=128 * _log(rng, 1, 112), dtype=rng.choice(["f32", "bf16"]))
        elif op == "quant_cols":
            case = dict(op=op, R=_log(rng, 1, 131072), C=16 * _log(rng, 1, 896), E=_log(rng, 1, 256),
                        skew=rng.choice([0.0, 1.0, 1.2]), dtype=rng.choice(["f32", "bf16"]))
        elif op == "quant_weights":
            tr = rng.random() < 0.5
            a, b = 16 * _log(rng, 1, 1792), 128 * _log(rng, 1, 112)
            case = dict(op=op, E=_log(rng, 1, 64), N=b if tr else a, K=a if tr else b, transposed=tr)
        elif op == "gemm":
            case = dict(op=op, R=_log(rng, 1, 131072), E=_log(rng, 1, 64), N=16 * _log(rng, 8, 1792),
                        K=128 * _log(rng, 1, 112), skew=rng.choice([0.0, 1.0, 1.2]), out=rng.choice(["bf16", "f32"]))
        else:
            case = dict(op=op, R=_log(rng, 16, 131072), E=_log(rng, 1, 64), N=16 * _log(rng, 8, 896),
                        K=16 * _log(rng, 8, 896), skew=rng.choice([0.0, 1.0, 1.2]), out=rng.choice(["bf16", "f32"]))
        # outputs and weights of at most 4 GB, so that a state fits three times over
        big = case.get("E", 1) * case.get("N", 1) * case.get("K", 1) <= 5e8 and case.get("R", 1) * case.get("N", 1) <= 1e9
        if _fits(case) and big:
            return case


def _torch_dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def work(case):
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        lg = T * E * (4 if case["dtype"] == "f32" else 2)
        mask = T if case["masked"] else 0
        if op == "route_fwd":
            return {"bytes": lg + mask + T * k * 8 + 4 * E + 8, "flops": T * E * 5}
        return {"bytes": 2 * lg + mask + T * k * 12 + 4 * E + 8, "flops": T * E * 8}
    if op in ("quant_rows", "quant_cols"):
        n = case["R"] * case["C"]
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + 1) + n // 32, "flops": 3 * n}
    E, N, K = case["E"], case["N"], case["K"]
    if op == "quant_weights":
        return {"bytes": E * N * K * 3 + E * N * K // 4096, "flops": 3 * E * N * K}
    R = case["R"]
    flops, osz = 2.0 * R * N * K, 4 if case["out"] == "f32" else 2
    if op == "wgrad":
        return {"bytes": R * (N + K) + R * (N + K) // 32 + E * N * K * osz, "flops": flops}
    pop = [(e + 1) ** -case["skew"] for e in range(E)]
    hit = sum(1 - (1 - p / sum(pop)) ** R for p in pop)   # experts that have a row at all
    return {"bytes": R * K + R * K // 32 + hit * N * K + R * N * osz, "flops": flops}


# ---------------------------------------------------------------------------- inputs

def _counts(gen, R, E, skew):
    """Rows of each expert: R draws, popularity (e + 1)^-skew in an order of its own."""
    pop = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-skew)
    pop = pop[torch.randperm(E, generator=gen, device="cuda")]
    ids = torch.multinomial(pop / pop.sum(), R, replacement=True, generator=gen)
    return torch.bincount(ids, minlength=E)


def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


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
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal(gen, (T, E), 1.5, _torch_dtype(case["dtype"]))
        s["mask"] = None
        if case["masked"]:   # sequences end in padding tokens, which do not count
            s["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.85
        if op == "route_bwd":
            idx, prob, counts, _ = _route(s["logits"], k, s["mask"])
            s.update(idx=idx, prob=prob, counts=counts, dprob=torch.randn((T, k), generator=gen, device="cuda") / T,
                     dlosses=torch.tensor([0.01, 0.001], device="cuda"))
        return s
    if op == "quant_rows":
        s["x"] = _activations(gen, case["R"], case["C"], _torch_dtype(case["dtype"]))
        return s
    if op == "quant_cols":
        s["offsets"] = _offsets(_counts(gen, case["R"], case["E"], case["skew"]))
        s["x"] = _activations(gen, case["R"], case["C"], _torch_dtype(case["dtype"]))
        return s
    E, N, K = case["E"], case["N"], case["K"]
    if op == "quant_weights":
        s["w"] = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            s["w"][e] = _normal(gen, (N, K), 0.02)
        return s
    R = case["R"]
    counts = _counts(gen, R, E, case["skew"])
    s["offsets"] = _offsets(counts)
    s["counts"] = counts.tolist()     # the host's copy, which the plain form loops over
    if op == "gemm":
        s["a"], s["a_scales"] = _quant_rows(_activations(gen, R, K, torch.bfloat16))
        s["w"] = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
        s["w_scales"] = torch.empty((E, -(-N // 128), K // 128), device="cuda")
        for e in range(E):
            s["w"][e], s["w_scales"][e] = _quant_matrix(_normal(gen, (N, K), 0.02))
    else:
        s["dyt"], s["dyt_scales"] = _quant_cols(_activations(gen, R, N, torch.bfloat16) * 0.01, s["offsets"])
        s["xt"], s["xt_scales"] = _quant_cols(_activations(gen, R, K, torch.bfloat16), s["offsets"])
    return s


# ---------------------------------------------------------------------------- plain forms

def _scales(amax):
    """fp32 (quantization factor, scale) of a block's largest magnitude: 448 / amax and amax / 448,
    both kept to normal numbers; a block of zeros has 1 and 1."""
    factor = (E4M3_MAX / amax).clamp(max=1 / TINY)
    scale = (amax / E4M3_MAX).clamp(min=TINY)
    none = amax == 0
    return torch.where(none, torch.ones_like(factor), factor), torch.where(none, torch.ones_like(scale), scale)


def _quant_rows(x):
    """codes [R, C] and scales [C / 128, R]."""
    R, C = x.shape
    v = x.float().view(R, C // 128, 128)
    factor, scale = _scales(v.abs().amax(2))
    return (v * factor[:, :, None]).to(F8).view(torch.uint8).view(R, C), scale.t().contiguous()


def _quant_matrix(w):
    """codes [N, K] and scales [ceil(N / 128), K / 128] of 128 x 128 blocks; the last rows may be fewer."""
    N, K = w.shape
    nb = -(-N // 128)
    v = torch.zeros((nb * 128, K), device=w.device)
    v[:N] = w
    factor, scale = _scales(v.view(nb, 128, K // 128, 128).abs().amax((1, 3)))
    v = v.view(nb, 128, K // 128, 128) * factor[:, None, :, None]
    return v.to(F8).view(torch.uint8).view(nb * 128, K)[:N], scale


def _quant_cols(x, offsets):
    """codes [C, P] and scales [P / 128, C]: every expert's rows padded with zeros to whole blocks of 128."""
    R, C = x.shape
    E = offsets.numel() - 1
    P = -(-R // 128) * 128 + 128 * E
    o = offsets.long()
    padded = -(-(o[1:] - o[:-1]) // 128) * 128
    starts = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    at = torch.arange(P, device=x.device)
    e = (torch.searchsorted(starts, at, right=True) - 1).clamp(max=E - 1)
    src = o[e] + at - starts[e]
    live = src < o[e + 1]
    v = torch.where(live[:, None], x[src.clamp(max=R - 1)].float(), 0.0).view(P // 128, 128, C)
    factor, scale = _scales(v.abs().amax(1))
    codes = (v * factor[:, None, :]).to(F8).view(torch.uint8)
    return codes.view(P, C).t().contiguous(), scale


def _route(logits, k, mask):
    """Top-k ids (ties: lowest id), their softmax weights, per-expert counts and [balance loss, z-loss]."""
    T, E = logits.shape
    v = logits.float()
    val, idx = torch.sort(v, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    w = torch.exp(val - val[:, :1])
    prob = w / w.sum(1, keepdim=True)
    top = v.amax(1, keepdim=True)
    ex = torch.exp(v - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, (top + torch.log(total))[:, 0]
    live = torch.ones(T, device=v.device, dtype=torch.bool) if mask is None else mask
    counts = torch.bincount(idx.reshape(-1), weights=live[:, None].expand(T, k).reshape(-1).double(), minlength=E)
    n = live.sum().double().clamp(min=1)
    psum = torch.where(live[:, None], p, 0.0).sum(0, dtype=torch.float64)
    balance = E / (k * n * n) * (counts * psum).sum()
    z = torch.where(live, lse * lse, 0.0).sum(dtype=torch.float64) / n
    return idx.to(torch.int32), prob, counts.to(torch.int32), torch.stack([balance, z]).float()


def _route_bwd(logits, idx, prob, counts, dprob, dlosses, mask):
    T, E = logits.shape
    k = idx.shape[1]
    v = logits.float()
    top = v.amax(1, keepdim=True)
    ex = torch.exp(v - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, top + torch.log(total)
    n = (counts.sum().double() / k).clamp(min=1)
    f = (counts * (E / (k * n * n))).float()
    d = dlosses[0] * p * (f - (p * f).sum(1, keepdim=True)) + dlosses[1] * (2 / n).float() * lse * p
    if mask is not None:
        d = torch.where(mask[:, None], d, 0.0)
    dsel = prob * (dprob - (prob * dprob).sum(1, keepdim=True))
    d.scatter_add_(1, idx.long(), dsel)
    return d.to(logits.dtype)


def _values(codes, scales):
    """fp32 values of row codes [R, C] with scales [C / 128, R]."""
    R, C = codes.shape
    return (codes.view(F8).float().view(R, C // 128, 128) * scales.t()[:, :, None]).view(R, C)


def _matrix_values(codes, scales):
    N, K = codes.shape
    rows = scales.repeat_interleave(128, 0)[:N]
    return (codes.view(F8).float().view(N, K // 128, 128) * rows[:, :, None]).view(N, K)


def _gemm(s):
    a = _values(s["a"], s["a_scales"])
    out = torch.empty((s["R"], s["N"]), dtype=_torch_dtype(s["out"]), device=a.device)
    at = 0
    for e, m in enumerate(s["counts"]):   # one product for each expert that has rows
        if m:
            out[at:at + m] = a[at:at + m] @ _matrix_values(s["w"][e], s["w_scales"][e]).t()
            at += m
    return out


def _wgrad(s):
    dy, x = _values_t(s["dyt"], s["dyt_scales"]), _values_t(s["xt"], s["xt_scales"])
    out = torch.zeros((s["E"], s["N"], s["K"]), dtype=_torch_dtype(s["out"]), device=dy.device)
    at = 0
    for e, m in enumerate(s["counts"]):
        if m:
            out[e] = dy[:, at:at + m] @ x[:, at:at + m].t()
            at += -(-m // 128) * 128
    return out


def _values_t(codes, scales):
    """fp32 values of token-axis codes [C, P] with scales [P / 128, C]."""
    C, P = codes.shape
    return (codes.view(F8).float().view(C, P // 128, 128) * scales.t()[:, :, None]).view(C, P)


def _seen(codes, scales):
    return {"codes": codes.view(F8), "scales": scales}


def run(s):
    op = s["op"]
    if own:
        import mixture_experts_grouped_permute_amd as m
        if op == "route_fwd":
            idx, prob, counts, losses = m.moe_route_balance(s["logits"], s["k"], token_mask=s["mask"])
            return {"idx": idx, "prob": prob, "counts": counts, "losses": losses}
        if op == "route_bwd":
            return m.moe_route_balance_bwd(s["logits"], s["idx"], s["prob"], s["counts"], s["dprob"], s["dlosses"],
                                           token_mask=s["mask"])
        if op == "quant_rows":
            return _seen(*m.fp8_block_quantize(s["x"]))
        if op == "quant_cols":
            return _seen(*m.fp8_block_quantize(s["x"], axis=1, group_offsets=s["offsets"]))
        if op == "quant_weights":
            return _seen(*m.fp8_block_quantize_weights(s["w"], transposed=s["transposed"]))
        if op == "gemm":
            return m.fp8_block_grouped_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"],
                                            out_dtype=_torch_dtype(s["out"]))
        return m.fp8_block_grouped_wgrad(s["dyt"], s["dyt_scales"], s["xt"], s["xt_scales"], s["offsets"],
                                         out_dtype=_torch_dtype(s["out"]))
    if op == "route_fwd":
        idx, prob, counts, losses = _route(s["logits"], s["k"], s["mask"])
        return {"idx": idx, "prob": prob, "counts": counts, "losses": losses}
    if op == "route_bwd":
        return _route_bwd(s["logits"], s["idx"], s["prob"], s["counts"], s["dprob"], s["dlosses"], s["mask"])
    if op == "quant_rows":
        return _seen(*_quant_rows(s["x"]))
    if op == "quant_cols":
        return _seen(*_quant_cols(s["x"], s["offsets"]))
    if op == "quant_weights":
        return _seen(*_quant_weights(s["w"], s["transposed"]))
    return _gemm(s) if op == "gemm" else _wgrad(s)


def _quant_weights(w, transposed):
    E, N, K = w.shape
    rows, cols = (K, N) if transposed else (N, K)
    codes = torch.empty((E, rows, cols), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, -(-rows // 128), cols // 128), device=w.device)
    for e in range(E):   # one matrix at a time: fp32 copies of all of them would not fit beside each other
        codes[e], scales[e] = _quant_matrix(w[e].t() if transposed else w[e])
    return codes, scales


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definitions, in 64 bits; whole numbers and codes (whose rounding borders move with
    the last bit of a factor) have no such value."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        l = s["logits"].double()
        T, E, k = case["T"], case["E"], case["k"]
        p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
        live = (s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device="cuda")).double()
        n = max(1.0, float(live.sum()))
        order = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
        picked = torch.zeros_like(l).scatter_(1, order, 1.0)
        share = (picked * live[:, None]).sum(0) / (n * k)
        if op == "route_fwd":
            chosen = torch.softmax(torch.gather(l, 1, order), 1)
            mean = (p * live[:, None]).sum(0) / n
            losses = torch.stack([E * (share * mean).sum(), (lse.square() * live).sum() / n])
            return {"idx": None, "prob": chosen, "counts": None, "losses": losses}
        ids = s["idx"].long()
        sel = s["prob"].double()
        g = s["dprob"].double()
        gb, gz = s["dlosses"].double()
        grad = E * gb / n * live[:, None] * (p * share - p * (p * share).sum(1, keepdim=True))
        grad = grad + gz * 2 / n * live[:, None] * lse[:, None] * p
        return grad + torch.zeros_like(grad).scatter_(1, ids, sel * g - sel * (sel * g).sum(1, keepdim=True))
    if op == "quant_rows":
        amax = s["x"].double().view(case["R"], -1, 128).abs().amax(2).t()
        return {"codes": None, "scales": torch.where(amax > 0, amax / 448, 1.0)}
    if op == "quant_cols":
        rows, lim = [], s["offsets"].tolist()
        P = -(-case["R"] // 128) + case["E"]
        for lo, hi in zip(lim[:-1], lim[1:]):
            for b in range(lo, hi, 128):
                rows.append(s["x"][b:min(hi, b + 128)].abs().amax(0).double() / 448)
        scales = torch.ones((P, case["C"]), dtype=torch.float64, device="cuda")
        if rows:
            scales[:len(rows)] = torch.where(torch.stack(rows) > 0, torch.stack(rows), 1.0)
        return {"codes": None, "scales": scales}
    if op == "quant_weights":
        out = []
        for w in s["w"]:
            m = w.t() if case["transposed"] else w
            pad = -m.shape[0] % 128
            m = torch.nn.functional.pad(m.abs(), (0, 0, 0, pad)).reshape(-1, 128, m.shape[1] // 128, 128)
            out.append(m.amax((1, 3)).double() / 448)
        return {"codes": None, "scales": torch.stack(out)}
    lim = s["offsets"].tolist()
    if op == "gemm":
        out = torch.zeros((case["R"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            lo, hi = lim[e], lim[e + 1]
            if hi == lo:
                continue
            a = s["a"][lo:hi].view(F8).double()
            a *= s["a_scales"][:, lo:hi].double().t().repeat_interleave(128, 1)
            w = s["w"][e].view(F8).double()
            w *= s["w_scales"][e].double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:case["N"]]
            out[lo:hi] = a @ w.t()
        return out
    out = torch.zeros((case["E"], case["N"], case["K"]), dtype=torch.float64, device="cuda")
    b0 = 0
    for e in range(case["E"]):
        nb = -(-(lim[e + 1] - lim[e]) // 128)
        if nb:
            both = []
            for c, sc in (("dyt", "dyt_scales"), ("xt", "xt_scales")):
                v = s[c][:, b0 * 128:(b0 + nb) * 128].contiguous().view(F8).double()
                both.append(v * s[sc][b0:b0 + nb].double().t().repeat_interleave(128, 1))
            out[e] = both[0] @ both[1].t()
        b0 += nb
    return out

"""GPU parity of the block-scaled FP8 operators against the numpy oracle.

Quantization: codes and scales bit for bit.  Products, with S = sum of the magnitudes of the scaled
products of an output, B its number of blocks of 128 and u = 2^-24:
  * fp32 output: E4M3 products are exact in the bf16 matrix instructions; 4 chained sums per block, the
    scale product and the running sum round: (2 B + 16) u S;
  * bf16 output: half a bf16 step of the value, 2^-8 |v|, and the E4M3 instructions' alignment, which
    drops what is below 2^-16 of the largest of a group of products -- at most 8 of them: 2^-13 S.
"""
import numpy as np
import pytest
import torch

from gpu_util import gpu, log, need_gpu
from oracle import block

U = 2.0 ** -24


def _x(shape, dtype, seed, spread=4):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * np.exp2(g.integers(-spread, spread + 1, shape[-1:]))
    t = torch.from_numpy(x).to(torch.bfloat16)
    if dtype == torch.float32:
        t = t.float() * (1 + torch.from_numpy(g.uniform(0, 1e-3, shape)).float())
    return t


def _np(t):
    return t.cpu().float().numpy()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 384), (31, 512), (33, 640), (257, 1408), (64, 4096)])
def test_quantize_rows(rows, cols, dtype):
    m = need_gpu()
    x = _x((rows, cols), dtype, rows + cols)
    x[0, :128] = 0.0
    if rows > 2:
        x[1, :128] = torch.linspace(-1e-38, 1e-38, 128).to(dtype)      # scale at its floor
        x[2, 5] = -0.0
        x[2, 6] = float(torch.finfo(dtype).max)
    q, s = m.fp8_block_quantize(x.cuda())
    torch.cuda.synchronize()
    rq, rs = block.quantize_rows(_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


SEGS = [("one", [5], 16), ("exact-blocks", [128, 256], 128), ("ragged", [0, 1, 127, 0, 129, 300, 0], 144),
        ("many", [17] * 70 + [0] * 3 + [400], 272), ("empty-tail", [200, 0, 0], 1040)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,cols", SEGS, ids=[c[0] for c in SEGS])
def test_quantize_tokens(name, sizes, cols, dtype):
    m = need_gpu()
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    x = _x((int(off[-1]), cols), dtype, cols)
    x[:, 3] = 0.0
    q, s = m.fp8_block_quantize(x.cuda(), axis=1, group_offsets=torch.from_numpy(off).cuda())
    torch.cuda.synchronize()
    rq, rs = block.quantize_tokens(_np(x), off)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    if len(sizes) == 1:
        q2, s2 = m.fp8_block_quantize(x.cuda(), axis=1)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@gpu
def test_quantize_tokens_bad_offsets_stay_inside():
    """Decreasing and out-of-range offsets are clamped; every output byte is written all the same."""
    m = need_gpu()
    x = _x((300, 64), torch.bfloat16, 1).cuda()
    for off in ([0, 500, 100, 300], [-5, 200, 100, 1 << 30], [0, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        q, s = m.fp8_block_quantize(x, axis=1, group_offsets=o)
        torch.cuda.synchronize()
        top = np.maximum.accumulate(np.clip(off, 0, 300))
        rq, rs = block.quantize_tokens(_np(x), top)
        np.testing.assert_array_equal(q.cpu().numpy(), rq)
        np.testing.assert_array_equal(s.cpu().numpy(), rs)


@gpu
@pytest.mark.parametrize("E,rows,cols", [(1, 16, 128), (3, 128, 256), (2, 144, 384), (70, 256, 128), (2, 384, 1408)])
def test_quantize_weights_both_ways(E, rows, cols):
    m = need_gpu()
    w = _x((E, rows, cols), torch.bfloat16, E)
    w[0, :16, :128] = 0.0
    q, s = m.fp8_block_quantize_weights(w.cuda())
    wt = w.transpose(1, 2).contiguous()                    # [E, cols, rows]: rows of wt are the product's K
    qt, st = m.fp8_block_quantize_weights([t.cuda() for t in wt], transposed=True)
    torch.cuda.synchronize()
    for e in range(E):
        rq, rs = block.quantize_matrix(_np(w[e]))
        np.testing.assert_array_equal(q[e].cpu().numpy(), rq)
        np.testing.assert_array_equal(s[e].cpu().numpy(), rs)
    assert torch.equal(q, qt) and torch.equal(s, st)
    skip = torch.ones(E, dtype=torch.int32)
    skip[0] = 0
    q2, s2 = m.fp8_block_quantize_weights(w.cuda(), skip=skip.cuda())
    assert not q2[0].any() and not s2[0].any() and torch.equal(q2[1:], q[1:]) and torch.equal(s2[1:], s[1:])


@gpu
def test_blocks_with_infinity_or_nan_decode_to_nothing_finite():
    m = need_gpu()
    x = torch.ones((4, 256), dtype=torch.float32)
    x[0, 3] = float("inf")
    x[1, 200] = float("nan")
    q, s = m.fp8_block_quantize(x.cuda())
    v = q.view(torch.float8_e4m3fn).float().cpu().view(4, 2, 128) * s.cpu().t()[:, :, None]
    assert not torch.isfinite(v[0, 0]).any() and not torch.isfinite(v[1, 1]).any()
    assert torch.equal(v[0, 1], torch.ones(128)) and torch.equal(v[1, 0], torch.ones(128))


# sizes (rows per expert), N, K
GEMM = [
    ("single-token", [1], 16, 128),
    ("decode", [0, 1, 0, 3, 1, 0, 2, 1], 256, 512),
    ("decode-wide", [2, 0, 5, 1], 2816, 2048),
    ("seventeen", [17, 0, 16, 15], 272, 384),
    ("ragged", [0, 33, 255, 0, 257, 1], 400, 256),
    ("one-block", [300, 129], 128, 128),
    ("tall", [2000, 1, 700], 528, 640),
    ("experts-70", [3] * 40 + [0] * 10 + [60] * 20, 144, 256),
    # long K: tiles split along it, few rows (parts of 3 blocks or more) and full tiles (18 or more)
    ("split-few-rows", [3, 0, 9], 400, 8192),
    ("split-one-row", [0, 0, 1], 48, 4224),
    ("split-full-tiles", [600, 0, 40], 400, 5120),
    ("split-last-round", [256, 200, 0, 256], 256 * 23, 4736),
    ("split-29-rows", [20, 0, 9], 400, 8192),
    ("split-two-rounds", [25], 128 * 140, 2048),
    # few rows an expert: several groups of one expert, K's blocks uneven among the waves, a last odd column
    # fragment, every column width
    ("few-crowded", [35, 0, 0, 0, 1], 144, 640),
    ("few-sixteen", [16], 48, 384),
    ("few-wide", [0, 3, 17] * 20 + [0, 60], 1040, 896),
    ("few-one-block", [1, 0, 2] * 50, 336, 128),
]


def _gemm_inputs(m, sizes, N, K, seed=11):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    a, s = m.fp8_block_quantize(_x((int(off[-1]), K), torch.bfloat16, seed).cuda())
    w, ws = m.fp8_block_quantize_weights((_x((len(sizes), N, K), torch.bfloat16, seed + 1) * 0.05).cuda())
    return off, a, s, w, ws


def _check(got, ref, mag, blocks, dtype):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = (2 * blocks + 16) * U * mag if dtype == torch.float32 else 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K", GEMM, ids=[c[0] for c in GEMM])
def test_grouped_gemm(name, sizes, N, K, dtype):
    m = need_gpu()
    log(f"block gemm {name} {dtype}")
    off, a, s, w, ws = _gemm_inputs(m, sizes, N, K)
    out = m.fp8_block_grouped_gemm(a, s, w, ws, torch.from_numpy(off).cuda(), out_dtype=dtype)
    torch.cuda.synchronize()
    assert out.dtype == dtype
    ref, mag = block.grouped_gemm(a.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(), off)
    _check(out, ref, mag, K // 128, dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R", [9, 700])
def test_grouped_gemm_leaves_rows_outside_the_offsets(R, dtype):
    m = need_gpu()
    off, a, s, w, ws = _gemm_inputs(m, [R], 144, 256)
    w, ws = w.repeat(3, 1, 1), ws.repeat(3, 1, 1)
    full = m.fp8_block_grouped_gemm(a, s, w[:1].contiguous(), ws[:1].contiguous(), torch.from_numpy(off).cuda(),
                                    out_dtype=dtype)
    for o in ([2, 2, R // 2, R - 3], [0, R + 50, 5, R], [-4, 3, 1, 6], [5, 5, 5, 5]):
        out = torch.full((R, 144), 7.0, dtype=dtype, device="cuda")
        m.fp8_block_grouped_gemm(a, s, w, ws, torch.tensor(o, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()
        top = np.maximum.accumulate(np.clip(o, 0, R))
        lo, hi = int(top[0]), int(top[-1])
        assert (out[:lo] == 7).all() and (out[hi:] == 7).all()
        assert torch.allclose(out[lo:hi].float(), full[lo:hi].float(), rtol=2.0 ** -7, atol=1e-6 + 1e-4 * float(full.abs().max()))


@gpu
def test_grouped_gemm_nan_rows_stay_alone():
    """A row whose scale or codes are not finite, and the bytes behind the last row, reach no other row."""
    m = need_gpu()
    for sizes in ([5, 3], [300, 100]):
        off, a, s, w, ws = _gemm_inputs(m, sizes, 144, 256)
        o = torch.from_numpy(off).cuda()
        ref = m.fp8_block_grouped_gemm(a, s, w, ws, o)
        a2, s2 = a.clone(), s.clone()
        s2[0, 1] = float("nan")
        s2[1, sizes[0]] = float("inf")
        a2[2, 7] = 0x7F
        out = m.fp8_block_grouped_gemm(a2, s2, w, ws, o)
        torch.cuda.synchronize()
        bad = torch.zeros(sum(sizes), dtype=torch.bool, device="cuda")
        bad[[1, 2, sizes[0]]] = True
        assert torch.equal(out[~bad], ref[~bad]) and not torch.isfinite(out[bad]).all(dim=1).any()


@gpu
def test_dgrad_is_the_product_with_transposed_weights():
    m = need_gpu()
    sizes, N, K = [200, 0, 77], 256, 384
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    w = (_x((3, N, K), torch.bfloat16, 5) * 0.05).cuda()
    dy, s = m.fp8_block_quantize(_x((277, N), torch.bfloat16, 6).cuda())
    wt, wts = m.fp8_block_quantize_weights(w, transposed=True)
    dx = m.fp8_block_grouped_gemm(dy, s, wt, wts, torch.from_numpy(off).cuda(), out_dtype=torch.float32)
    wq, wqs = m.fp8_block_quantize_weights(w)
    torch.cuda.synchronize()
    vals = np.stack([block.values_matrix(wq[e].cpu().numpy(), wqs[e].cpu().numpy()) for e in range(3)])
    dyv = block.values_rows(dy.cpu().numpy(), s.cpu().numpy())
    ref = np.concatenate([dyv[off[e]:off[e + 1]] @ vals[e] for e in range(3)])
    mag = np.concatenate([np.abs(dyv[off[e]:off[e + 1]]) @ np.abs(vals[e]) for e in range(3)])
    _check(dx, ref, mag, N // 128, torch.float32)


WGRAD = [("tiny", [1], 16, 16), ("ragged", [0, 1, 127, 0, 129, 300, 0], 144, 272), ("blocks", [256, 128], 256, 128),
         ("wide", [700, 50], 528, 400), ("experts-70", [3] * 40 + [0] * 10 + [60] * 20, 48, 80),
         ("none", [0, 0, 4], 32, 32), ("split-tokens", [5000, 10, 0, 900], 48, 80),
         ("split-full-tiles", [6000, 1], 272, 400)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K", WGRAD, ids=[c[0] for c in WGRAD])
def test_grouped_wgrad(name, sizes, N, K, dtype):
    m = need_gpu()
    log(f"block wgrad {name} {dtype}")
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    o = torch.from_numpy(off).cuda()
    dyt, ds = m.fp8_block_quantize(_x((int(off[-1]), N), torch.bfloat16, 3).cuda(), axis=1, group_offsets=o)
    xt, xs = m.fp8_block_quantize(_x((int(off[-1]), K), torch.bfloat16, 4).cuda(), axis=1, group_offsets=o)
    out = torch.full((len(sizes), N, K), float("nan"), dtype=dtype, device="cuda")
    m.fp8_block_grouped_wgrad(dyt, ds, xt, xs, o, out=out)
    torch.cuda.synchronize()
    ref, mag = block.grouped_wgrad(dyt.cpu().numpy(), ds.cpu().numpy(), xt.cpu().numpy(), xs.cpu().numpy(), off)
    for e, n in enumerate(sizes):
        if n == 0:
            assert not out[e].any()
    _check(out, ref, mag, -(-max(sizes) // 128), dtype)


@gpu
def test_wgrad_bad_offsets_stay_inside():
    m = need_gpu()
    dyt = torch.full((32, 512), 0x38, dtype=torch.uint8, device="cuda")
    xt = torch.full((48, 512), 0x38, dtype=torch.uint8, device="cuda")
    ds, xs = torch.ones((4, 32), device="cuda"), torch.ones((4, 48), device="cuda")
    for off, want in (([0, 600, 100, 700], [512.0, 0.0, 0.0]), ([-3, 100, 300, 1 << 30], [128.0, 256.0, 128.0])):
        dw = m.fp8_block_grouped_wgrad(dyt, ds, xt, xs, torch.tensor(off, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        for e in range(3):
            assert (dw[e] == want[e]).all()


@gpu
def test_products_in_graphs_and_on_streams():
    m = need_gpu()
    runs = []
    # few rows, whole tiles, tiles split along K, along the tokens
    for sizes, N, K in (([4, 0, 2], 512, 512), ([300, 40, 513], 400, 384), ([20, 0, 9], 400, 8192),
                        ([5000, 10, 0, 900], 48, 128)):
        off, a, s, w, ws = _gemm_inputs(m, sizes, N, K)
        o = torch.from_numpy(off).cuda()
        xt = m.fp8_block_quantize(_x((int(off[-1]), 64), torch.bfloat16, 4).cuda(), axis=1, group_offsets=o)
        for dt in (torch.bfloat16, torch.float32):
            runs.append(lambda a=a, s=s, w=w, ws=ws, o=o, dt=dt: m.fp8_block_grouped_gemm(a, s, w, ws, o, out_dtype=dt))
            runs.append(lambda x=xt, o=o, dt=dt: m.fp8_block_grouped_wgrad(*x, *x, o, out_dtype=dt))
    want = [f() for f in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, f in enumerate(runs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(f())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs, outs = [], []
    for half in (runs[:4], runs[4:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs += [f() for f in half]
        graphs.append(g)
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(runs[0](), want[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@gpu
def test_block_refusals_on_the_gpu():
    m = need_gpu()
    x = torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.MoeError):
        m.fp8_block_quantize(x[:, :192].contiguous())
    with pytest.raises(ValueError):
        m.fp8_block_quantize(x[:, :128])                       # not contiguous
    with pytest.raises(ValueError):
        m.fp8_block_quantize(x, group_offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        m.fp8_block_quantize(x.half())
    off, a, s, w, ws = _gemm_inputs(m, [4, 4], 128, 256)
    o = torch.from_numpy(off).cuda()
    with pytest.raises(ValueError):
        m.fp8_block_grouped_gemm(a, s.t().contiguous(), w, ws, o)
    with pytest.raises(ValueError):
        m.fp8_block_grouped_gemm(a, s, w, ws, o[:2].contiguous())
    with pytest.raises(TypeError):
        m.fp8_block_grouped_gemm(a, s, w, ws, o.long())
    with pytest.raises(TypeError):
        m.fp8_block_grouped_gemm(a, s, w, ws, o, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        m.fp8_block_grouped_gemm(a, s, w, ws, o, out=torch.empty((8, 64), device="cuda"))
    qa, sa = m.fp8_block_quantize(x, axis=1, group_offsets=o)
    with pytest.raises(ValueError):
        m.fp8_block_grouped_wgrad(qa, sa, qa, sa[:2].contiguous(), o)


# both sides of the limit on products of few rows, over all 256 experts
FEW_LIMIT = [("few-512", [2] * 250 + [0] * 4 + [5, 7], 272, 640), ("tiles-768", [3] * 250 + [0] * 4 + [11, 7], 272, 640),
             ("tiles-crowded", [0] * 100 + [520] + [0] * 155, 272, 640)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K", FEW_LIMIT, ids=[c[0] for c in FEW_LIMIT])
def test_grouped_gemm_of_many_experts(name, sizes, N, K, dtype):
    test_grouped_gemm(name, sizes, N, K, dtype)


# More tiles than the persistent grid's 256 workgroups, in either output type: workgroups take a second and third
# tile, whole rounds are followed by a split one, the weight gradient's rounds alternate in direction.
GEMM_ROUNDS = [
    ("two-rounds", [4500], 4144, 384),                     # 306 tiles (fp32: 594)
    ("round-then-split", [4500], 4144, 2560),              # the last 50 (82) in two parts each
    ("partial-then-split", [(7 * i) % 41 for i in range(30)], 2320, 1024),   # edges of few rows, 4 parts
    ("join-walk-bf16", [2560], 2000, 2560),                # 80 split tiles of 32 row groups: the join's
    ("join-walk-f32", [2560], 1008, 2560),                 # 2048 workgroups go round, past an odd last column
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K", GEMM_ROUNDS, ids=[c[0] for c in GEMM_ROUNDS])
def test_grouped_gemm_of_several_rounds(name, sizes, N, K, dtype):
    test_grouped_gemm(name, sizes, N, K, dtype)


WGRAD_ROUNDS = [
    ("rounds", [700, 0, 129, 300, 1], 1040, 2816),         # 275 tiles (fp32: 550) of 0 to 6 blocks
    ("rounds-then-split", [385 + (i * 53) % 400 for i in range(130)], 16, 512),   # the last 4 (8) in two parts each
]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name,sizes,N,K", WGRAD_ROUNDS, ids=[c[0] for c in WGRAD_ROUNDS])
def test_grouped_wgrad_of_several_rounds(name, sizes, N, K, dtype):
    test_grouped_wgrad(name, sizes, N, K, dtype)

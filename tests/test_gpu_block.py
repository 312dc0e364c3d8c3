"""Block operators on the GPU against the float64 oracle.

Tolerances are error bounds, not fits.  u(t) = eps(t) / 2 is one rounding to
type t.  Norm: the sum of squares of a row takes at most 16 additions in a
thread, 5 in a warp and 32 over warps, with a few roundings around it:
under 64 FP32 roundings, 2^-18.  Routing weights: exp of a difference of at
most 24 (24 roundings), the sum (21) and a few more: under 64, 2^-18.
Linear: FP32 accumulation over K/16 steps of the tensor core (which may
truncate, 2^-23 a step) and the sum of at most 8 parts: (K/16 + 16) 2^-23 of
the sum of |products|; activations have slopes of at most 1.13.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from w4a16_compact_expert_gb300 import block as B
from w4a16_compact_expert_gb300 import moe_w4a16 as F

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}   # half a smallest step
N32 = 2.0 ** -18


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


# ------------------------------------------------------------------ add_rmsnorm
def check_norm(x, res, w, eps, outs):
    y, s, q, qs = outs
    rs, rn = O.add_rmsnorm(f64(x), None if res is None else f64(res), None if w is None else f64(w), eps)
    dt = x.dtype
    if y is not None:
        assert (np.abs(f64(y) - rn) <= (U[dt] + N32) * np.abs(rn) * 1.01 + TINY[dt]).all()
    if s is not None:
        assert (np.abs(f64(s) - rs) <= (U[dt] + 2.0 ** -23) * np.abs(rs) + TINY[dt]).all()
    if q is not None:
        ref = np.abs(rn).max(-1) / 448
        assert (np.abs(f64(qs) - ref) <= N32 * ref).all()
        c = f64(qs)[:, None]
        ok = c[:, 0] > 0
        v = rn[ok] / c[ok]
        assert (np.abs(f64(q.float())[ok] - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2.0 ** -10)).all()
        assert (f64(q.float())[~ok] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (5, 130), (2, 2048), (67, 2047), (33, 2052), (9, 4096),
                                 (3, 8191), (2, 8200), (9, 12289), (9, 16383), (3, 16384),
                                 (1000, 256), (129, 72), (37, 40), (41, 9), (8, 1023)])
def test_norm_shapes(T, H, dtype):
    x, res, w = rand((T, H), dtype, 1), rand((T, H), dtype, 2, 3.0), rand((H,), dtype, 3)
    for r, ww, quant in ((res, w, True), (None, w, True), (res, None, False), (None, None, False)):
        outs = B.add_rmsnorm(x, r, ww, quant=quant)
        assert (outs[1] is None) == (r is None) and (outs[2] is None) == (not quant)
        check_norm(x, r, ww, 1e-6, outs)


@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_norm_strides_and_alignment(off):
    T, H = 11, 520
    big = rand((T, H + 24), torch.float16, 5)
    x = big[:, off:off + H]
    res = rand((T, H + 8), torch.float16, 6)[:, :H]
    w = rand((H + 8,), torch.float16, 7)[off:off + H]
    guard = torch.full((T, H + 16), 7.0, dtype=torch.float16, device="cuda")
    s = torch.full((T, H + 16), 7.0, dtype=torch.float16, device="cuda")
    q = torch.zeros((T, H + 16), device="cuda").to(torch.float8_e4m3fn)
    qs = torch.empty(T, device="cuda")
    outs = B.add_rmsnorm(x, res, w, quant=True, out=(guard[:, off:off + H], s[:, :H], q[:, off:off + H], qs))
    check_norm(x, res, w, 1e-6, outs)
    assert (guard[:, :off] == 7).all() and (guard[:, off + H:] == 7).all() and (s[:, H:] == 7).all()
    assert (q.float()[:, :off] == 0).all() and (q.float()[:, off + H:] == 0).all()


@pytest.mark.parametrize("T,H", [(5000, 1024), (4003, 1030), (3000, 2056), (2501, 4097), (2600, 8192), (2440, 9001),
                                 (2433, 16384)])
def test_norm_many_rows(T, H):
    """Enough rows for the streaming kernel, every row against the direct kernel's and some against the oracle."""
    for dtype, r, quant in ((torch.float16, True, True), (torch.bfloat16, False, False)):
        x, w = rand((T, H), dtype, 1), rand((H,), dtype, 3)
        res = rand((T, H), dtype, 2) if r else None
        outs = B.add_rmsnorm(x, res, w, quant=quant)
        pick = [0, 1, 2, T // 2, T - 2, T - 1]
        cut = lambda t: None if t is None else t[pick]   # noqa: E731
        check_norm(x[pick], cut(res), w, 1e-6, [cut(o) for o in outs])
        for i in range(0, T, 500):   # the direct kernel's rows: within the roundings of two summation orders
            few = B.add_rmsnorm(x[i:i + 500], None if res is None else res[i:i + 500], w)[0]
            d = (few.double() - outs[0][i:i + 500].double()).abs()
            assert (d <= 2.5 * U[dtype] * few.double().abs() + 2 * TINY[dtype]).all()


def test_norm_in_place_and_rows_independent_of_batch():
    x, res, w = rand((300, 2048), torch.float16, 8), rand((300, 2048), torch.float16, 9), rand((2048,), torch.float16, 10)
    y, s, q, qs = B.add_rmsnorm(x, res, w, quant=True)
    x2, r2 = x.clone(), res.clone()
    B.add_rmsnorm(x2, r2, w, quant=True, out=(x2, r2, torch.empty_like(q), torch.empty_like(qs)))
    assert torch.equal(x2, y) and torch.equal(r2, s)
    y1, s1, q1, qs1 = B.add_rmsnorm(x[17:18], res[17:18], w, quant=True)
    assert torch.equal(y1[0], y[17]) and torch.equal(q1.view(torch.uint8)[0], q.view(torch.uint8)[17]) and qs1[0] == qs[17]


def test_norm_zero_tiny_and_nonfinite_rows():
    x = rand((6, 320), torch.bfloat16, 11)
    x[0] = 0
    x[1] = 1e-38
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 0
    x[4, 319] = 2.0
    y, _, q, qs = B.add_rmsnorm(x, quant=True, eps=0.0)
    assert torch.isnan(y[2]).any() and torch.isnan(y[3]).any()
    y, _, q, qs = B.add_rmsnorm(x, quant=True)
    assert (y[0] == 0).all() and (q.float()[0] == 0).all() and qs[0] == 0
    assert torch.isnan(q.float()[2, 5]) and torch.isnan(q.float()[3, 7])
    keep = [0, 1, 4, 5]
    check_norm(x[keep], None, None, 1e-6, (y[keep], None, q[keep], qs[keep]))


def test_norm_no_rows():
    y, s, q, qs = B.add_rmsnorm(torch.empty(0, 64, dtype=torch.float16, device="cuda"), quant=True)
    assert y.shape == (0, 64) and q.shape == (0, 64) and qs.shape == (0,)


# ------------------------------------------------------------------ route_scored
def check_route(logits, bias, k, **kw):
    ids, w = B.route_scored(logits, k, bias=bias, **kw)
    rid, rw = O.route_scored(f64(logits), None if bias is None else f64(bias), k, **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(f64(w) - rw) <= N32 * np.abs(rw) + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,rank", [
    (1, 1, 1, 1, 1, 1), (5, 8, 2, 1, 1, 1), (9, 60, 4, 1, 1, 2), (33, 64, 8, 1, 1, 1), (40, 64, 6, 8, 3, 2),
    (17, 160, 6, 8, 3, 1), (8, 100, 32, 1, 1, 1), (50, 256, 8, 8, 4, 2), (7, 300, 10, 5, 2, 2), (6, 512, 16, 32, 7, 2),
    (4, 96, 3, 32, 1, 1), (12, 20, 20, 1, 1, 1), (3, 6, 2, 3, 2, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(T, E, k, groups, top_groups, rank, score, biased, dtype):
    logits = rand((T, E), dtype, E + T, 1.5)
    bias = rand((E,), torch.float32, 3, 0.1) if biased else None
    for renorm, scale in ((False, 1.0), (True, 2.5)):
        check_route(logits, bias, k, score=score, groups=groups, top_groups=top_groups, group_rank=rank,
                    renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_borders_closer_than_fp32(score):
    """Choices that differ by less than FP32 scores resolve: biases undo the
    differences of the scores, computed in 64 bits and rounded to FP32."""
    T, E, k = 64, 64, 8
    logits = rand((1, E), torch.float32, 21, 1.0).expand(T, E).clone()
    l = f64(logits[0])
    sc = np.exp(l - l.max()) / np.exp(l - l.max()).sum() if score == "softmax" else 1 / (1 + np.exp(-l))
    bias = torch.from_numpy((1.0 - sc).astype(np.float32)).cuda()   # every choice is 1 within 2^-25
    ids, _ = check_route(logits, bias, k, score=score)
    fp32 = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    assert not torch.equal(torch.sort(fp32 + bias, dim=-1, descending=True, stable=True)[1][:, :k].int(), ids)
    for groups, top in ((8, 3), (4, 2)):
        check_route(logits, bias, k, score=score, groups=groups, top_groups=top, group_rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(64, 8, 1, 1), (64, 8, 8, 4), (256, 8, 8, 4), (60, 6, 6, 3), (30, 5, 1, 1)])
def test_route_a_few_close_borders(score, E, k, groups, top):
    """Pairs and triples of choices (and of group values) that FP32 cannot order, at every place of the order."""
    T = 96
    g = torch.Generator().manual_seed(E + k + groups)
    logits = torch.randn(T, E, generator=g)
    l = logits[0].double()
    sc = (torch.softmax(l, -1) if score == "softmax" else torch.sigmoid(l)).numpy()
    per = E // groups
    want = np.linspace(1.0, 2.0, E)                       # choices far apart ..
    np.random.default_rng(E).shuffle(want)
    order = np.argsort(-want)
    for r in range(0, E - 2, 3):                          # .. except every second and third of the order
        want[order[r + 1]] = want[order[r]]
        if r % 2:
            want[order[r + 2]] = want[order[r]]
    if groups > 1:                                        # groups 1 and 2 hold the same two largest choices
        a, b = np.argsort(-want[per:2 * per])[:2] + per, np.argsort(-want[2 * per:3 * per])[:2] + 2 * per
        want[b] = want[a]
    bias = torch.from_numpy((want - sc).astype(np.float32)).cuda()   # back to `want` within a rounding of FP32
    logits[:] = logits[0]
    logits[1::2] += torch.randn(T // 2, E, generator=g) * 1e-6       # and rows a little off it
    check_route(logits.cuda(), bias, k, score=score, groups=groups, top_groups=top, group_rank=2 if per > 1 else 1)
    check_route(logits.cuda(), bias, k, score=score, groups=groups, top_groups=top, group_rank=1, renormalize=True)


def test_route_close_groups_without_a_bias():
    """Group sums that FP32 cannot order: two groups hold the same logits but for the last bits."""
    T, E = 64, 64
    logits = rand((T, E), torch.float32, 51)
    logits[:, 8:16] = logits[:, 0:8] * (1 + 2.0 ** -23)
    logits[:, 16:24] = logits[:, 0:8].flip(1)
    for score in ("softmax", "sigmoid"):
        for top in (1, 2, 3):
            check_route(logits, None, 4, score=score, groups=8, top_groups=top, group_rank=2)


def test_route_ties_go_to_the_lower_index():
    logits = torch.zeros(7, 96, device="cuda")
    logits[1] = torch.arange(96, device="cuda") % 3
    logits[2, 40:] = -0.0
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.full((96,), 0.25, device="cuda")):
            ids, _ = check_route(logits, bias, 9, score=score, groups=1)
            assert ids[0].tolist() == list(range(9)) and ids[2].tolist() == list(range(9))
            check_route(logits, bias, 9, score=score, groups=8, top_groups=3, group_rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_masks(score, biased, groups, top):
    E, k = 32, 6
    logits = rand((8, E), torch.float32, 31)
    inf = float("inf")
    logits[0] = -inf                      # nothing left
    logits[1, 1:] = -inf                  # one expert left
    logits[2, ::2] = float("nan")         # half masked by NaN
    logits[3, :] = float("nan")
    logits[4, 8:] = -inf                  # one group left
    logits[5] = torch.finfo(torch.float32).min
    logits[6, 3] = 300.0                  # underflow of all others
    logits[7] = -200.0                    # sigmoids below FP32
    logits[7, 5] = -199.0
    bias = rand((E,), torch.float32, 32, 0.1) if biased else None
    if biased:
        bias[9] = -inf
        bias[10] = float("nan")
    for renorm in (False, True):
        ids, w = check_route(logits, bias, k, score=score, groups=groups, top_groups=top, group_rank=2,
                             renormalize=renorm)
        assert ids[0].tolist() == list(range(k)) and (w[0] == 0).all() and (w[3] == 0).all()
        assert torch.isfinite(w).all()
        for row in ids.tolist():
            assert len(set(row)) == k


def test_route_strided_logits():
    big = rand((19, 100), torch.float16, 41)
    check_route(big[:, 3:67], None, 8, renormalize=True)


def test_route_many_tokens():
    logits = rand((5000, 64), torch.float32, 43, 0.9)
    bias = rand((64,), torch.float32, 44, 0.05)
    check_route(logits, bias, 8, score="sigmoid", groups=8, top_groups=4, group_rank=2, renormalize=True, scale=2.5)


# ------------------------------------------------------------------ linear
def make_linear(T, N, K, dtype, act, bias, residual, out_dtype, seed=0):
    M = 2 * N if act == "swiglu" else N
    x, w = rand((T, K), torch.float32, seed + 1), rand((M, K), torch.float32, seed + 2, 1.0 / K ** 0.5)
    xs = ws = None
    if dtype is torch.float8_e4m3fn:
        xs, ws = x.abs().amax(-1) / 448, w.abs().amax(-1) / 448
        x, w = (x / xs[:, None]).to(dtype), (w / ws[:, None]).to(dtype)
    else:
        x, w = x.to(dtype), w.to(dtype)
    b = rand((M,), torch.float32, seed + 3) if bias else None
    r = rand((T, N), out_dtype, seed + 4) if residual else None
    return x, w, xs, ws, b, r


def check_linear(x, w, xs, ws, b, r, act, out, r_in=None):
    g = lambda t: None if t is None else f64(t.float())   # noqa: E731
    ref, pre, mag = O.linear(g(x), g(w), g(xs), g(ws), g(b), act, g(r) if r_in is None else r_in)
    err = (x.shape[1] / 16 + 16) * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(pre)
    if act == "swiglu":
        n = w.shape[0] // 2
        gate, up, eg, eu = pre[:, :n], pre[:, n:], err[:, :n], err[:, n:]
        sl = np.abs(O.silu(gate))
        err = 1.13 * eg * (np.abs(up) + eu) + sl * eu + 2.0 ** -20 * np.abs(ref)
    else:
        err = 1.13 * err + 2.0 ** -20 * np.abs(pre)
    tol = U[out.dtype] * (np.abs(ref) + err) + err + TINY[out.dtype] + 2.0 ** -24 * np.abs(ref)
    got = f64(out)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(got - ref).max()))


F16, BF16, F32, E4 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("T,N,K", [(1, 1, 8), (1, 128, 64), (1, 300, 2048), (2, 129, 72), (15, 64, 2048), (16, 7, 128),
                                   (17, 256, 264), (31, 1000, 520), (33, 130, 1024), (64, 65, 200), (65, 512, 512),
                                   (127, 33, 4096), (128, 128, 8), (129, 257, 1000), (300, 200, 328), (513, 700, 160)])
@pytest.mark.parametrize("dtype,out", [(F16, F16), (BF16, BF16), (F16, F32)], ids=["fp16", "bf16", "fp32out"])
def test_linear_shapes(T, N, K, dtype, out):
    t = make_linear(T, N, K, dtype, "none", False, False, out, T)
    check_linear(*t, "none", B.linear(t[0], t[1], out_dtype=out))


@pytest.mark.parametrize("T", [1, 16, 30, 61, 100])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("N,K", [(4096, 3000), (12000, 1536), (20, 20000)])
def test_linear_every_pipeline_stage(T, act, N, K):
    """Enough K chunks per CTA to go round the ring, with few and many tiles."""
    for dtype in (F16, E4):
        t = make_linear(T, N, K // 16 * 16, dtype, act, False, False, F16, T)
        x, w, xs, ws, _, _ = t
        check_linear(*t, act, B.linear(x, w, act=act, x_scale=xs, w_scale=ws, out_dtype=F16))


@pytest.mark.parametrize("T,N,K,act", [(1100, 9000, 208, "none"), (1100, 9000, 256, "gelu"), (2000, 4100, 144, "swiglu"),
                                       (1500, 4097, 512, "swiglu"), (260, 20000, 176, "none"), (4000, 300, 1040, "silu")])
def test_linear_wide_many_tiles(T, N, K, act):
    """More tiles than resident CTAs, rows on and off 128-byte lines, every output."""
    for dtype in (F16, E4):
        t = make_linear(T, N, K, dtype, act, True, False, F16, T)
        x, w, xs, ws, b, _ = t
        check_linear(*t, act, B.linear(x, w, act=act, bias=b, x_scale=xs, w_scale=ws, out_dtype=F16))


@pytest.mark.parametrize("T,N,K", [(1, 100, 16), (5, 64, 2048), (40, 129, 272), (130, 300, 1024)])
@pytest.mark.parametrize("out", [F16, BF16, F32], ids=["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_e4m3(T, N, K, out, act):
    t = make_linear(T, N, K, E4, act, True, True, out, N)
    x, w, xs, ws, b, r = t
    check_linear(*t, act, B.linear(x, w, bias=b, act=act, residual=r, x_scale=xs, w_scale=ws, out_dtype=out))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("T", [1, 20, 200])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_linear_epilogue(act, T, bias, residual):
    for dtype, out, N in ((F16, F16, 190), (BF16, BF16, 61), (F16, F32, 64)):
        t = make_linear(T, N, 384, dtype, act, bias, residual, out, T)
        x, w, _, _, b, r = t
        check_linear(*t, act, B.linear(x, w, bias=b, act=act, residual=r, out_dtype=out))


@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_linear_strides_guards_and_in_place_residual(T, off):
    N, K = 150, 96
    x = rand((T, K + 40), F16, 1)[:, 8:8 + K]
    w = rand((N, K + 8), F16, 2, 0.1)[:, :K]
    buf = torch.full((T + 1, N + 30), 3.0, dtype=F16, device="cuda")
    out = buf[:T, off:off + N]
    check_linear(x, w, None, None, None, None, "none", B.linear(x, w, out=out))
    assert (buf[T] == 3).all() and (buf[:, :off] == 3).all() and (buf[:, off + N:] == 3).all()
    res = rand((T, N), F16, 3)
    keep = f64(res)
    got = B.linear(x, w, residual=res, act="gelu", out=res)
    assert got.data_ptr() == res.data_ptr()
    check_linear(x, w, None, None, None, None, "gelu", got, r_in=keep)


@pytest.mark.parametrize("dtype", [F16, BF16, E4], ids=["fp16", "bf16", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 1, 1001), (1, 130, 1001), (2, 1, 33), (17, 65, 77), (70, 129, 1001)])
def test_linear_odd_k_and_single_rows(dtype, T, N, K):
    """K off the 16-byte grid (rows padded to it), and single rows of x or W, whose stride counts for nothing."""
    x, w, xs, ws, b, r = make_linear(T, N, K, dtype, "none", True, True, F32)
    padded = []
    for t in (x, w):
        p = torch.full((t.shape[0], (K + 15) // 16 * 16), 7.0, device="cuda").to(dtype)   # never read as values
        p[:, :K] = t
        padded.append(p[:, :K] if t.shape[0] > 1 else p[0, :K].view(1, K))
    x, w = padded
    check_linear(x, w, xs, ws, b, r, "none",
                 B.linear(x, w, x_scale=xs, w_scale=ws, bias=b, residual=r, out_dtype=F32))
    if N > 1:   # no rows of x at all
        none = B.linear(x[:0], w, x_scale=None if xs is None else xs[:0], w_scale=ws, out_dtype=F32)
        assert none.shape == (0, N)


def test_linear_same_result_every_run_and_nothing_left_over():
    """Runs twice over several splits; a large-valued call in between must leave no trace."""
    for T, N, K in ((1, 64, 4096), (16, 512, 2048), (100, 300, 1024), (400, 260, 512)):
        x, w, *_ = make_linear(T, N, K, F16, "none", False, False, F16)
        a = B.linear(x, w)
        B.linear(x * 60, w * 60)
        assert torch.equal(a, B.linear(x, w))
    assert B.status() == F.OK


def test_linear_masked_and_nonfinite_values():
    x, w, *_ = make_linear(4, 130, 80, F16, "none", False, False, F16)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    out = B.linear(x, w)
    assert torch.isnan(out[2]).all() and not torch.isfinite(out[1]).any()
    check_linear(x[[0, 3]], w, None, None, None, None, "none", out[[0, 3]])
    assert torch.isnan(B.linear(x, w, act="relu")[2]).all()
    one = torch.ones(1, 8, dtype=F16, device="cuda")
    big = torch.tensor([[6e4, 0, 0, 0, 0, 0, 0, 0]] * 2, device="cuda").half() * torch.tensor([[1.0], [-1.0]], device="cuda").half()
    for act in ("gelu", "gelu_tanh", "silu"):   # far out the activations are a and 0, not NaN
        got = B.linear(one, big, act=act, out_dtype=F32)[0]
        assert got[0] == big[0, 0].float() and got[1].abs() < 1e-3, act


def test_linear_no_rows():
    x, w, *_ = make_linear(1, 130, 80, F16, "none", False, False, F16)
    assert B.linear(x[:0], w).shape == (0, 130)


def test_operators_on_a_stream_and_in_a_graph():
    x, res, w = rand((24, 512), F16, 1), rand((24, 512), F16, 2), rand((512,), F16, 3)
    rw = rand((64, 512), F16, 4, 0.05)
    wd = rand((512, 512), F16, 5, 0.05)

    def chain():
        y, s, _, _ = B.add_rmsnorm(x, res, w)
        ids, gw = B.route_scored(B.linear(y, rw, out_dtype=F32), 8, renormalize=True)
        return B.linear(y, wd, act="silu", residual=s), ids, gw

    ref = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    x.copy_(rand((24, 512), F16, 9))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, chain()))
    y = B.add_rmsnorm(x, res, w, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, B.add_rmsnorm(x, res, w)[0])
    assert B.status() == F.OK

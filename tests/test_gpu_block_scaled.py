"""The block-scaled 8-bit path on the GPU against the float64 oracle.

Tolerances are error bounds, not fits.  u(t) = eps(t) / 2 is one rounding to
type t.  Norm: under 64 FP32 roundings, 2^-18 (as the norm with a scale per
row); a scale adds two.  Linear: a block of 128 takes 4 steps of the tensor core
(which may truncate, 2^-23 a step) and one for its sum over them, is scaled (one
rounding of the scale) and added (one): (kb + 16) 2^-23 of the sum of |products|
over kb blocks, the sum of at most 8 parts included; activations have slopes of
at most 1.13.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from w4a16_compact_expert_gb300 import block as B
from w4a16_compact_expert_gb300 import moe_w4a16 as F

pytestmark = pytest.mark.gpu

F16, BF16, F32, E4 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}   # half a smallest step
N32 = 2.0 ** -18


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def check_quantised(q, qs, ref, rel):
    """q qs against ref [T, n], whose values the kernel knows to rel (relative): the scales, then every value to half
    a step of E4M3 at its place on the scale that was given."""
    s = O.block_scales(ref)
    assert (np.abs(f64(qs) - s) <= (rel + 2.0 ** -22) * s + 2.0 ** -126).all()
    c = np.repeat(f64(qs), 128, -1)[:, :ref.shape[1]]
    got, ok = f64(q.float()), c > 0
    v = np.divide(ref, c, out=np.zeros_like(ref), where=ok)
    # the value v carries rel and two roundings of the division before it is rounded
    assert (np.abs(got - v)[ok] <= (np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2.0 ** -10) + (rel + 2.0 ** -21) * np.abs(v))[ok]).all()
    assert (got[~ok] == 0).all()


# ------------------------------------------------------------------ add_rmsnorm
def check_norm(x, res, w, eps, outs):
    y, s, q, qs = outs
    rs, rn = O.add_rmsnorm(f64(x), None if res is None else f64(res), None if w is None else f64(w), eps)
    dt = x.dtype
    if y is not None:
        assert (np.abs(f64(y) - rn) <= (U[dt] + N32) * np.abs(rn) * 1.01 + TINY[dt]).all()
    if s is not None:
        assert (np.abs(f64(s) - rs) <= (U[dt] + 2.0 ** -23) * np.abs(rs) + TINY[dt]).all()
    check_quantised(q, qs, rn, N32)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 64), (40, 120), (5, 127), (5, 128), (70, 129), (5, 136), (9, 256),
                                 (33, 264), (2, 2048), (67, 2047), (33, 2056), (9, 4096), (3, 8191), (2, 8200), (9, 12288),
                                 (9, 16383), (3, 16384), (1000, 256), (129, 72), (41, 9), (8, 1023)])
def test_norm_shapes(T, H, dtype):
    x, res, w = rand((T, H), dtype, 1), rand((T, H), dtype, 2, 3.0), rand((H,), dtype, 3)
    for r, ww, norm in ((res, w, True), (None, w, True), (res, None, False), (None, None, False)):
        outs = B.add_rmsnorm(x, r, ww, norm=norm, quant="blocks")
        assert (outs[0] is None) == (not norm) and (outs[1] is None) == (r is None)
        assert outs[3].shape == (T, -(-H // 128))
        check_norm(x, r, ww, 1e-6, outs)


@pytest.mark.parametrize("T,H", [(5000, 1024), (4003, 1032), (3000, 2056), (2501, 4097), (2600, 8192), (2440, 9000),
                                 (2433, 16384)])
def test_norm_many_rows(T, H):
    """Enough rows for the streaming kernel; y and s are the bits of the norm with a scale per row where both take the
    same path (rows on the 16-byte grid)."""
    for dtype, r in ((F16, True), (BF16, False)):
        x, w = rand((T, H), dtype, 1), rand((H,), dtype, 3)
        res = rand((T, H), dtype, 2) if r else None
        outs = B.add_rmsnorm(x, res, w, quant="blocks")
        pick = [0, 1, 2, T // 2, T - 2, T - 1]
        cut = lambda t: None if t is None else t[pick]   # noqa: E731
        check_norm(x[pick], cut(res), w, 1e-6, [cut(o) for o in outs])
        if H % 8 == 0:
            y, s, _, _ = B.add_rmsnorm(x, res, w)
            assert torch.equal(y, outs[0]) and (not r or torch.equal(s, outs[1]))
        n = outs[0].float()   # the scales of every row, from the rounded norm
        nb = -(-H // 128)
        ref = torch.nn.functional.pad(n, (0, nb * 128 - H)).view(T, nb, 128).abs().amax(-1) / 448
        assert ((outs[3] - ref).abs() <= 1.01 * U[dtype] * ref + 2.0 ** -24).all()


@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_norm_strides_and_alignment(off):
    T, H = 11, 520
    x = rand((T, H + 24), F16, 5)[:, off:off + H]
    res = rand((T, H + 8), F16, 6)[:, :H]
    w = rand((H + 8,), F16, 7)[off:off + H]
    guard = torch.full((T, H + 16), 7.0, dtype=F16, device="cuda")
    s = torch.full((T, H + 16), 7.0, dtype=F16, device="cuda")
    q = torch.zeros((T, H + 16), device="cuda").to(E4)
    qs = torch.full((T + 2, 5), 7.0, device="cuda")
    outs = B.add_rmsnorm(x, res, w, quant="blocks", out=(guard[:, off:off + H], s[:, :H], q[:, off:off + H], qs[1:T + 1]))
    check_norm(x, res, w, 1e-6, outs)
    assert (guard[:, :off] == 7).all() and (guard[:, off + H:] == 7).all() and (s[:, H:] == 7).all()
    assert (q.float()[:, :off] == 0).all() and (q.float()[:, off + H:] == 0).all()
    assert (qs[0] == 7).all() and (qs[T + 1] == 7).all()


def test_norm_zero_blocks_and_nonfinite_rows():
    x = rand((6, 320), BF16, 11)
    x[0] = 0
    x[1, 128:256] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 0
    x[4, 319] = 2.0
    y, _, q, qs = B.add_rmsnorm(x, quant="blocks")
    assert (q.float()[0] == 0).all() and (qs[0] == 0).all() and qs[1, 1] == 0 and (q.float()[1, 128:256] == 0).all()
    assert torch.isnan(q.float()[2, 5]) and torch.isnan(q.float()[3, 7])
    keep = [0, 1, 4, 5]
    check_norm(x[keep], None, None, 1e-6, (y[keep], None, q[keep], qs[keep]))


def test_norm_refusals_and_no_rows():
    x = rand((4, 300), F16, 1)
    y, s, q, qs = B.add_rmsnorm(x[:0], quant="blocks")
    assert q.shape == (0, 300) and qs.shape == (0, 3)
    with pytest.raises(ValueError):
        B.add_rmsnorm(x, quant="rows")
    q, y = torch.empty(4, 300, device="cuda").to(E4), torch.empty_like(x)
    for bad in (torch.empty(4, device="cuda"), torch.empty(4, 2, device="cuda"), torch.empty(4, 3, device="cuda").half(),
                torch.empty(3, 4, device="cuda").t(), torch.empty(4, 6, device="cuda")[:, :3]):
        with pytest.raises(ValueError):
            B.add_rmsnorm(x, quant="blocks", out=(y, None, q, bad))


# ---------------------------------------------------------------- linear_blocks
def blocks(n):
    return -(-n // 128)


def make_linear(T, N, K, act="none", bias=False, residual=False, out=F16, seed=0):
    """Random E4M3 values with scales that differ by a factor of up to 16 between blocks."""
    M, parts = (2 * N, 2) if act == "swiglu" else (N, 1)
    g = torch.Generator().manual_seed(seed)
    scales = lambda r, c, std: (torch.exp2(torch.rand(r, c, generator=g) * 4 - 2) * std / 64).cuda()   # noqa: E731
    x, w = rand((T, K), F32, seed + 1, 64.0).to(E4), rand((M, K), F32, seed + 2, 64.0).to(E4)
    xs, ws = scales(T, blocks(K), 1.0), scales(parts * blocks(N), blocks(K), 0.05)
    b = rand((M,), F32, seed + 3) if bias else None
    r = rand((T, N), out, seed + 4) if residual else None
    return x, w, xs, ws, b, r


def reference(x, w, xs, ws, b, r, act, r_in=None):
    """(result in float64, how far a result in FP32 may be off)"""
    g = lambda t: None if t is None else f64(t.float())   # noqa: E731
    ref, pre, mag = O.linear_blocks(g(x), g(w), g(xs), g(ws), g(b), act, g(r) if r_in is None else r_in)
    err = (blocks(x.shape[1]) + 16) * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(pre)
    if act == "swiglu":
        n = w.shape[0] // 2
        gate, up, eg, eu = pre[:, :n], pre[:, n:], err[:, :n], err[:, n:]
        err = 1.13 * eg * (np.abs(up) + eu) + np.abs(O.silu(gate)) * eu + 2.0 ** -20 * np.abs(ref)
    else:
        err = 1.13 * err + 2.0 ** -20 * np.abs(pre)
    return ref, err


def check_linear(x, w, xs, ws, b, r, act, out, r_in=None):
    ref, err = reference(x, w, xs, ws, b, r, act, r_in)
    if isinstance(out, tuple):
        q, qs = (f64(o.float()) for o in out)
        s = O.block_scales(ref)
        es = O.block_scales(err)   # the largest error of a block, over 448
        assert qs.shape == s.shape and (np.abs(qs - s) <= es + 2.0 ** -21 * s + 2.0 ** -126).all()
        c = np.repeat(qs, 128, -1)[:, :ref.shape[1]]
        ok = c > 0
        v, e = (np.divide(t, c, out=np.zeros_like(t), where=ok) for t in (ref, err))
        tol = np.maximum(2.0 ** -4 * (np.abs(v) + e), 2.0 ** -10) * (1 + 2.0 ** -10) + e + 2.0 ** -20 * np.abs(v)
        assert (np.abs(q - v) <= tol)[ok].all() and (q[~ok] == 0).all()
        return
    tol = U[out.dtype] * (np.abs(ref) + err) + err + TINY[out.dtype] + 2.0 ** -24 * np.abs(ref)
    got = f64(out)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(got - ref).max()))


def run(t, act, **kw):
    x, w, xs, ws, b, r = t
    return B.linear_blocks(x, w, xs, ws, bias=b, act=act, residual=r, **kw)


@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 128, 128), (1, 300, 2048), (2, 129, 80), (15, 64, 2048), (16, 7, 128),
                                   (17, 256, 272), (31, 1000, 528), (33, 130, 1024), (64, 65, 208), (65, 512, 512),
                                   (127, 33, 4096), (128, 128, 16), (129, 257, 1008), (300, 200, 336), (513, 700, 160)])
@pytest.mark.parametrize("out", [F16, BF16, F32, E4], ids=["fp16", "bf16", "fp32", "e4m3"])
def test_linear_shapes(T, N, K, out):
    t = make_linear(T, N, K, seed=T)
    check_linear(*t, "none", run(t, "none", out_dtype=out))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("T", [1, 20, 50, 200])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_linear_epilogue(act, T, bias, residual):
    for out, N in ((F16, 190), (BF16, 61), (F32, 64), (E4, 300), (E4, 128)):
        res = residual and out != E4
        t = make_linear(T, N, 384, act, bias, res, out, T)
        check_linear(*t, act, run(t, act, out_dtype=out))


@pytest.mark.parametrize("T", [1, 16, 30, 61, 100])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("N,K", [(4096, 3008), (12000, 1536), (20, 20000)])
def test_linear_every_pipeline_stage(T, act, N, K):
    """Enough K chunks per CTA to go round the ring, with few and many tiles."""
    t = make_linear(T, N, K, act, seed=T)
    check_linear(*t, act, run(t, act))


@pytest.mark.parametrize("T,N,K,act", [(1100, 9000, 208, "none"), (1100, 9000, 256, "gelu"), (2000, 4100, 144, "swiglu"),
                                       (1500, 4097, 512, "swiglu"), (260, 20000, 176, "none"), (4000, 300, 1040, "silu"),
                                       (3000, 4096, 128, "none"), (3000, 4096, 112, "swiglu"), (700, 2600, 2064, "none")])
def test_linear_wide_many_tiles(T, N, K, act):
    """More tiles than resident CTAs, one K block and many, every output."""
    for out in (F16, F32, E4):
        t = make_linear(T, N, K, act, True, False, out, T)
        check_linear(*t, act, run(t, act, out_dtype=out))


@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("off", [0, 1, 4, 16])
def test_linear_strides_guards_and_in_place_residual(T, off):
    N, K = 150, 272
    x0, w0, xs0, ws0, b, _ = make_linear(T, N, K, bias=True, seed=off)

    def padded(t, left, right, fill):
        p = torch.full((t.shape[0] + 2, left + t.shape[1] + right), fill, device="cuda").to(t.dtype)
        p[1:-1, left:left + t.shape[1]] = t
        return p[1:-1, left:left + t.shape[1]]

    x, w = padded(x0, 16, 48, 7.0), padded(w0, 32, 16, 7.0)
    xs, ws = padded(xs0, off % 4, 3, float("nan")), padded(ws0, 1, off, float("nan"))
    for out in (F16, F32, E4):
        buf = torch.full((T + 2, N + 40), 3.0, device="cuda").to(out)
        o = buf[1:T + 1, off:off + N]
        got = B.linear_blocks(x, w, xs, ws, bias=b, out=o)
        check_linear(x, w, xs, ws, b, None, "none", got)
        fence = buf.float()
        assert (fence[[0, T + 1]] == 3).all() and (fence[:, :off] == 3).all() and (fence[:, off + N:] == 3).all()
    res = rand((T, N), F16, 3)
    keep = f64(res)
    got = B.linear_blocks(x, w, xs, ws, residual=res, act="gelu", out=res)
    assert got.data_ptr() == res.data_ptr()
    check_linear(x, w, xs, ws, None, None, "gelu", got, r_in=keep)


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 1, 1001), (1, 130, 1001), (2, 1, 33), (17, 65, 77), (70, 129, 1001)])
def test_linear_odd_k_and_single_rows(T, N, K):
    """K off the 16-byte grid (rows padded to it), and single rows of x or W, whose stride counts for nothing."""
    x, w, xs, ws, b, r = make_linear(T, N, K, bias=True, residual=True, out=F32)
    pad = []
    for t in (x, w):
        p = torch.full((t.shape[0], (K + 15) // 16 * 16), 7.0, device="cuda").to(E4)   # never read as values
        p[:, :K] = t
        pad.append(p[:, :K] if t.shape[0] > 1 else p[0, :K].view(1, K))
    t = (*pad, xs, ws, b, r)
    check_linear(*t, "none", run(t, "none", out_dtype=F32))
    none = B.linear_blocks(t[0][:0], t[1], xs[:0], ws)
    assert none.shape == (0, N)
    q, s = B.linear_blocks(t[0][:0], t[1], xs[:0], ws, out_dtype=E4)
    assert q.shape == (0, N) and s.shape == (0, blocks(N))


@pytest.mark.parametrize("T", [3, 90])
def test_linear_zero_and_nonfinite_scales(T):
    """Zero scales take a block out; NaN and infinite ones stay with their token or their weight block."""
    x, w, xs, ws, _, _ = make_linear(T, 300, 512, seed=T)
    xs[0] = 0
    xs[1, 2] = 0
    ws[1, 0] = 0
    for out in (F16, E4):
        check_linear(x, w, xs, ws, None, None, "none", B.linear_blocks(x, w, xs, ws, out_dtype=out))
    q, s = B.linear_blocks(x, w, xs, ws, out_dtype=E4)
    assert (q.float()[0] == 0).all() and (s[0] == 0).all()
    xs[2, 1] = float("nan")
    out = B.linear_blocks(x, w, xs, ws, out_dtype=F32)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all() and torch.isfinite(out[3:]).all()
    q, s = B.linear_blocks(x, w, xs, ws, out_dtype=E4)
    assert torch.isnan(q.float()[2]).all() and torch.isfinite(q.float()[:2]).all()
    xs[2, 1] = 1.0
    ws[2, 3] = float("inf")
    out = B.linear_blocks(x, w, xs, ws, out_dtype=F32)
    assert torch.isfinite(out[:, :256]).all() and not torch.isfinite(out[1:, 256:]).any()


def test_linear_small_blocks_of_the_output():
    """Blocks of an E4M3 output that are zero, or too small for a scale."""
    for T in (4, 80):
        x, w, xs, ws, _, _ = make_linear(T, 384, 256, seed=T)
        ws[1] = 0
        ws[2] *= 1e-38
        q, s = B.linear_blocks(x, w, xs, ws, out_dtype=E4)
        assert (s[:, 1:] == 0).all() and (q.float()[:, 128:] == 0).all() and (s[:, 0] > 0).all()


def test_linear_same_result_every_run_streams_and_graphs():
    for T, N, K, act, out in ((1, 64, 4096, "none", F32), (16, 512, 2048, "swiglu", E4), (50, 300, 1024, "none", F16),
                              (100, 300, 1024, "swiglu", E4), (400, 260, 512, "none", F16)):
        t = make_linear(T, N, K, act, seed=1)
        get = lambda **kw: (lambda o: o if isinstance(o, tuple) else (o,))(run(t, act, out_dtype=out, **kw))   # noqa: E731
        same = lambda p, q: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(p, q))   # noqa: E731
        ref = get()
        B.linear_blocks(t[0], t[1], t[2] * 1e4, t[3] * 1e4, act=act, out_dtype=out)
        assert same(ref, get())
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = get()
        named = get(stream=side)
        side.synchronize()
        assert same(ref, other) and same(ref, named)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = get()
        t[0].copy_(make_linear(T, N, K, act, seed=7)[0])
        g.replay()
        torch.cuda.synchronize()
        assert same(got, get())
    assert B.status() == F.OK


def test_linear_refusals():
    x, w, xs, ws, b, _ = make_linear(4, 200, 256)
    ok = B.linear_blocks(x, w, xs, ws)
    q = torch.empty(4, 200, device="cuda").to(E4)
    for args, kw in (((x.half(), w, xs, ws), {}), ((x, w.half(), xs, ws), {}), ((x, w, xs[:, :1], ws), {}),
                     ((x, w, xs[:3], ws), {}), ((x, w, xs, ws[:1]), {}), ((x, w, xs.double(), ws), {}),
                     ((x, w[:, :128], xs, ws), {}), ((x, w, xs.t().contiguous().t(), ws), {}),
                     ((x, w, None, None), {}), ((x, w, xs, ws), dict(act="tanh")), ((x, w, xs, ws), dict(bias=torch.zeros(100, device="cuda"))),
                     ((x, w[:199], xs, ws), dict(act="swiglu")), ((x, w, xs, ws), dict(out_scale=xs)),
                     ((x, w, xs, ws), dict(out=q, residual=q.clone())), ((x, w, xs, ws), dict(out=q, out_scale=xs[:, :1])),
                     ((x, w, xs, ws), dict(out=q, out_dtype=F16)), ((x, w, xs, ws), dict(out=ok[:, :100])),
                     ((x, w, xs, ws), dict(residual=ok.float())), ((x[:, 8:], w[:, 8:], xs, ws), {}),
                     ((x, w, xs, ws.cpu()), {})):
        with pytest.raises((ValueError, F.MoEError)):
            B.linear_blocks(*args, **kw)


def test_offsets_past_32_bits():
    """The last rows of W and of the output where they take more than 2^31 and 2^32 bytes."""
    N, K = (1 << 22) + 200, 512
    w = torch.zeros(N, K, dtype=torch.uint8, device="cuda").view(E4)
    t = make_linear(130, 200, K, seed=3)
    w[N - 200:] = t[1]   # N - 200 is a multiple of 128: the blocks are the small problem's
    ws = torch.ones(blocks(N), blocks(K), device="cuda")
    ws[-2:] = t[3]
    x, xs = t[0], t[2]
    for T in (3, 130):
        out = torch.empty((1 << 32) // (2 * N) + 600, N, dtype=F16, device="cuda")[-T:]
        got = B.linear_blocks(x[:T], w, xs[:T], ws, out=out)
        check_linear(x[:T], t[1], xs[:T], t[3], None, None, "none", got[:, N - 200:])
        assert (got[:, :1000] == 0).all()


# ------------------------------------------------------------------ together
def test_norm_head_and_scores_together():
    """norm with a block-scaled copy -> output head -> log probabilities, each against the oracle on what it was given."""
    T, H, V = 37, 512, 5003
    x, res, w = rand((T, H), BF16, 1), rand((T, H), BF16, 2), rand((H,), BF16, 3)
    _, head, _, hs, _, _ = make_linear(1, V, H, seed=5)
    tok = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    y, s, q, qs = B.add_rmsnorm(x, res, w, quant="blocks")
    check_norm(x, res, w, 1e-6, (y, s, q, qs))
    logits = B.linear_blocks(q, head, qs, hs, out_dtype=F32)
    check_linear(q, head, qs, hs, None, None, "none", logits)
    p, e, ids, top = B.token_logprobs(logits, tok, 5)
    rp, re, rids, rtop, _ = O.token_logprobs(f64(logits), tok.cpu().numpy(), 5)
    assert np.array_equal(ids.cpu().numpy(), rids)
    for got, ref in ((p, rp), (e, re), (top, rtop)):
        assert (np.abs(f64(got) - ref) <= 2e-5 * (1 + np.abs(ref))).all()
    assert B.status() == F.OK


@pytest.mark.parametrize("T", [1, 33, 300])
def test_quantised_feed_forward(T):
    """gate and up with an E4M3 output, which down takes as it is: against the same in float64 from the given bits."""
    H, I = 512, 700
    x, gu, xs, gs, _, _ = make_linear(T, I, H, "swiglu", seed=T)
    _, down, _, ds, _, _ = make_linear(1, H, I // 16 * 16, seed=T + 1)
    down = torch.nn.functional.pad(down.view(torch.uint8), (0, 704 - down.shape[1])).view(E4)   # I off the 16-byte grid
    down[:, 696:] = 1.0
    out = torch.empty(T, 704, device="cuda").to(E4)
    h, hs = B.linear_blocks(x, gu, xs, gs, act="swiglu", out=out[:, :I])
    check_linear(x, gu, xs, gs, None, None, "swiglu", (h, hs))
    res = rand((T, H), F16, 9)
    keep = f64(res)
    got = B.linear_blocks(h, down[:, :I], hs, ds, residual=res, out=res)
    check_linear(h, down[:, :I], hs, ds, None, None, "none", got, r_in=keep)


@pytest.mark.parametrize("T,N,act", [(100, 272, "none"), (97, 144, "swiglu"), (257, 403, "none"), (70, 300, "swiglu"),
                                     (129, 31, "none"), (300, 129, "swiglu"), (66, 260, "gelu")])
def test_linear_e4m3_rows_of_any_layout(T, N, act):
    """The same bits whatever the distance and alignment of the output's rows, and nothing written beside them."""
    t = make_linear(T, N, 400, act, True, seed=N)
    want = None
    for ld, off in ((-(-N // 32) * 32, 0), (N, 0), (N + 16, 16), (N + 4 - N % 4, 4), (N + 1, 1), (N + 7, 3), (N + 36, 36)):
        buf = torch.full(((T + 2) * ld + 64,), 3.0, device="cuda").to(E4)
        o = buf[ld + off:].as_strided((T, N), (ld, 1))
        _, s = run(t, act, out=o)
        got = o.contiguous().view(torch.uint8)
        if want is None:
            want = (got, s)
            check_linear(*t, act, (o, s))
        assert torch.equal(got, want[0]) and torch.equal(s, want[1])
        o.view(torch.uint8).fill_(buf[:1].view(torch.uint8)[0])
        assert (buf.float() == 3).all()


@pytest.mark.parametrize("T", [1, 2, 90])
def test_outputs_fit_the_next_product_at_any_width(T):
    """Widths off the 16-byte grid: the E4M3 outputs that a call allocates are taken by the next as they are."""
    H, I = 300, 203
    pad = lambda t: torch.nn.functional.pad(t.view(torch.uint8), (0, -t.shape[1] % 16)).view(E4)[:, :t.shape[1]]   # noqa: E731
    x, w = rand((T, H), F16, 1), rand((H,), F16, 2)
    _, _, q, qs = B.add_rmsnorm(x, None, w, quant="blocks")
    _, gu, _, gs, _, _ = make_linear(1, I, H, "swiglu", seed=3)
    _, down, _, ds, _, _ = make_linear(1, H, I, seed=4)
    h, hs = B.linear_blocks(q, pad(gu), qs, gs, act="swiglu", out_dtype=E4)
    check_linear(q, gu, qs, gs, None, None, "swiglu", (h, hs))
    check_linear(h, down, hs, ds, None, None, "none", B.linear_blocks(h, pad(down), hs, ds))


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (9, 15), (50, 57), (4, 113), (4, 114), (6, 121), (17, 127), (9, 129),
                                 (33, 241), (33, 243), (5, 255), (5, 1001), (8, 2047), (4, 4095), (3, 8191), (2, 16383),
                                 (2433, 777), (2500, 1001), (2440, 2047), (2433, 5121), (2433, 10111), (2433, 16383)])
def test_norm_rows_off_the_grid(T, H):
    """Every place of a row on the 16-byte grid; only q elsewhere (the same sums, so the same bits); and all outputs
    elsewhere (another path, whose sums may have another order)."""
    for dtype, off, r in ((F16, 0, True), (BF16, 3, False), (F16, 7, True)):
        x, w = rand((T, H + off), dtype, 1), rand((H,), dtype, 3)
        x = x.view(-1)[off:off + T * H].view(T, H)
        res = rand((T, H + off), dtype, 2).view(-1)[off:off + T * H].view(T, H) if r else None
        flat = lambda t: torch.full((T * H + 16,), 3.0, device="cuda").to(t)[off:off + T * H].view(T, H)   # noqa: E731
        out = (flat(dtype), flat(dtype) if r else None, flat(E4), torch.empty(T, blocks(H), device="cuda"))
        B.add_rmsnorm(x, res, w, quant="blocks", out=out)
        pick = sorted({0, 1 % T, 2 % T, 3 % T, 4 % T, 5 % T, 6 % T, 7 % T, T // 2, T - 1})
        cut = lambda t: None if t is None else t[pick]   # noqa: E731
        check_norm(x[pick], cut(res), w, 1e-6, [cut(o) for o in out])
        check_norm(x[pick], cut(res), w, 1e-6, [cut(o) for o in B.add_rmsnorm(x, res, w, quant="blocks")])
        q = torch.zeros(T, H + 17 - H % 8, device="cuda").to(E4)[:, 1:H + 1]
        again = B.add_rmsnorm(x, res, w, quant="blocks", out=(flat(dtype), flat(dtype) if r else None, q, torch.empty_like(out[3])))
        assert torch.equal(out[0], again[0]) and torch.equal(out[3], again[3])
        assert torch.equal(out[2].view(torch.uint8), again[2].contiguous().view(torch.uint8))


def test_calls_on_several_streams_at_once():
    """Products of every form, norms and scores side by side, eagerly and from replayed graphs: each its own result."""
    jobs = []
    for i, (T, N, K, act, out) in enumerate(((300, 700, 1024, "swiglu", E4), (2000, 1000, 512, "none", F16), (8, 9000, 1024, "swiglu", E4),
                                             (60, 3000, 2048, "none", F32), (70, 2000, 640, "swiglu", BF16), (5, 30000, 512, "none", F32),
                                             (130, 100, 4096, "gelu", E4), (40, 600, 2992, "swiglu", F16))):
        t = make_linear(T, N, K, act, True, False, out, i)
        jobs.append(lambda t=t, act=act, out=out: run(t, act, out_dtype=out))
    x, w = rand((600, 2048), F16, 1), rand((2048,), F16, 2)
    a, b = rand((100, 4096), F16, 3), rand((3000, 4096), F16, 4, 0.02)
    lg, tok = rand((90, 40001), BF16, 5), torch.arange(90, device="cuda")
    jobs += [lambda: B.add_rmsnorm(x, None, w, quant="blocks"), lambda: B.linear(a, b), lambda: B.linear(a[:9], b),
             lambda: B.token_logprobs(lg, tok, 7)]
    bits = lambda r: [o.contiguous().view(torch.uint8) for o in (r if isinstance(r, tuple) else (r,)) if o is not None]   # noqa: E731
    ref = [bits(j()) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(6):
        for i, j in enumerate(jobs):
            with torch.cuda.stream(streams[(i + r) % 4]):
                got.append((i, j()))
    torch.cuda.synchronize()
    graphs = []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = [j() for j in jobs]
        graphs.append((g, outs))
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    got += [(i, o) for _, outs in graphs for i, o in enumerate(outs)]
    for i, o in got:
        assert all(torch.equal(p, q) for p, q in zip(bits(o), ref[i])), i
    from w4a16_compact_expert_gb300 import moe_w4a16 as F
    assert B.status() == F.OK

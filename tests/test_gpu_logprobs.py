"""token_logprobs on the GPU against the float64 oracle.

Tolerances are error bounds, u = 2^-24.  A term e^d, d = x - max: the
difference is off by u |d|, the product with log2 e by as much again, the
exponential by 2 ulp: 4 u |d| + 4 u relative.  The sum S: a thread adds V / 256
terms to a sum (two sums, 128 threads; one warp, up to 16 terms), with two
roundings per batch of 16 more, then three joins of six roundings and a
rescaling exponential of up to 4 u |d| + 4 u each, where what is rescaled far
weighs little:
  rel(S) <= (V / 256 + 150) u + 8 u D,   D = sum p |d|.
ln p: rel(S), the logarithm (2 ulp) and two subtractions: 4 u (|ln p| + ln V).
Entropy ln S - E / S: E's terms carry the same errors with weights p |d|:
  2 rel(S) (1 + D) + 8 u (D + D2) + 4 u ln V,   D2 = sum p d^2.
Ids are exact.
"""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from w4a16_compact_expert_gb300 import block as B
from w4a16_compact_expert_gb300 import moe_w4a16 as F

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
INF = math.inf
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(T, V, dtype, seed, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, V, generator=g, device="cuda") * std).to(dtype)


def tokens_of(T, V, seed, dtype=torch.int64):
    return torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def close(got, ref, tol):
    got = f64(got)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin])
    assert (np.abs(got - np.where(fin, ref, 0))[fin] <= np.broadcast_to(tol, ref.shape)[fin]).all()


def check(x, tok, k, outs):
    lp, ent, ids, top = outs
    T, V = x.shape
    rlp, rent, rids, rtop, sp = O.token_logprobs(f64(x), tok.cpu().numpy(), k)
    D, D2 = sp[:, 0], sp[:, 1]
    rs = (V / 256 + 150) * u + 8 * u * D
    lnv = math.log(V) + 1
    mag = lambda r: np.where(np.isfinite(r), np.abs(r), 0)   # noqa: E731
    close(lp, rlp, rs + 4 * u * (mag(rlp) + lnv))
    close(ent, rent, 2 * rs * (1 + D) + 8 * u * (D + D2) + 4 * u * lnv)
    if k:
        assert np.array_equal(ids.cpu().numpy(), rids)
        close(top, rtop, rs[:, None] + 4 * u * (mag(rtop) + lnv))
    else:
        assert ids is None and top is None


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V,k", [(1, 1, 0), (1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 31, 31), (3, 32, 32), (4, 33, 32),
                                   (7, 127, 5), (1, 129, 20), (65, 500, 20), (3, 1000, 1), (700, 1024, 8), (2, 4097, 32),
                                   (1, 8191, 20), (5, 8192, 32), (1, 9001, 32), (33, 16385, 7), (1, 32003, 20), (90, 32003, 5),
                                   (400, 20000, 4), (1300, 500, 16), (1300, 1000, 5), (1300, 3, 2), (1, 50304, 32), (40, 33000, 32), (17, 50304, 0), (2, 151936, 20), (1, 262145, 32)])
def test_shapes(T, V, k, dtype):
    x, tok = rand(T, V, dtype, V + k), tokens_of(T, V, T)
    check(x, tok, k, B.token_logprobs(x, tok, k))


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 33333), (9, 5003), (500, 777)])
@pytest.mark.parametrize("off", [0, 1, 3, 6])
def test_strides_and_alignment(T, V, off, dtype):
    big = rand(T, V + 11, dtype, off)
    big[:, :off] = 50.0   # never read as values
    big[:, off + V:] = 50.0
    x, tok = big[:, off:off + V], tokens_of(T, V, 1, torch.int32)
    check(x, tok, 16, B.token_logprobs(x, tok, 16))


def test_guards_of_the_outputs():
    T, V, k = 6, 700, 5
    x, tok = rand(T, V, torch.float32, 3), tokens_of(T, V, 4)
    f = torch.full((3, T + 2), 7.0, device="cuda")
    ids, top = torch.full((T + 2, k), -9, dtype=torch.int32, device="cuda"), torch.full((T + 2, k), 7.0, device="cuda")
    out = (f[0, 1:T + 1], f[1, 1:T + 1], ids[1:T + 1], top[1:T + 1])
    check(x, tok, k, B.token_logprobs(x, tok, k, out=out))
    assert (f[:, 0] == 7).all() and (f[:, T + 1] == 7).all() and (f[2] == 7).all()
    assert (ids[[0, T + 1]] == -9).all() and (top[[0, T + 1]] == 7).all()


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 40000), (12, 3001), (650, 300)])
def test_masks(T, V, dtype):
    """Masked shares up to rows with one, fewer than k and no value left, by -inf, NaN and the lowest finite value."""
    g = torch.Generator(device="cuda").manual_seed(V)
    low = torch.finfo(dtype).min
    for mask in (-INF, float("nan"), low):
        for keep in (0.5, 0.05, 3 / V, 1 / V, 0.0):
            x = rand(T, V, dtype, 5)
            x.masked_fill_(torch.rand(T, V, device="cuda", generator=g) >= keep, mask)
            if T > 4:
                x[1], x[2], x[3] = mask, mask, mask
                x[2, V - 1] = -3.0
                x[3, V // 2] = 1.0
            tok = tokens_of(T, V, 2)
            check(x, tok, 20, B.token_logprobs(x, tok, 20))


@pytest.mark.parametrize("T,V", [(1, 70001), (5, 2000), (610, 129)])
def test_ties_and_constant_rows(T, V):
    """Equal values go to the lower index, whatever part of the row they lie in."""
    for value in (0.0, -7.5, 1e-40, 65000.0):
        x = torch.full((T, V), value, device="cuda")
        x[:, V // 3] = -0.0 if value == 0.0 else value
        tok = tokens_of(T, V, 1)
        check(x, tok, 32, B.token_logprobs(x, tok, 32))
    g = torch.Generator(device="cuda").manual_seed(1)
    for levels in (2, 9, 50):
        x = torch.randint(0, levels, (T, V), device="cuda", generator=g).to(torch.bfloat16)
        x[:, ::2] *= -1
        tok = tokens_of(T, V, 1)
        check(x, tok, 17, B.token_logprobs(x, tok, 17))


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
def test_the_largest_crowd_in_few_places(dtype):
    """All large values within one window, one stride of threads, the row's ends, or ascending."""
    for T, V in ((1, 65536), (3, 20001), (400, 4500)):
        tok = tokens_of(T, V, 1)
        for case in range(5):
            x = rand(T, V, dtype, case, 0.1)
            big = rand(T, V, dtype, case + 9, 0.5) + 20
            if case == 0:
                x[:, 1000:1040] = big[:, 1000:1040]
            elif case == 1:
                x[:, ::512] = big[:, ::512]
            elif case == 2:
                x[:, :64] = big[:, :64]
                x[:, -3:] = big[:, -3:]
            elif case == 3:
                x = (torch.arange(V, device="cuda") / V * 60 - 30).to(dtype).expand(T, V).contiguous()
            else:
                x[:, 40:] = big[:, 40:]
            check(x, tok, 32, B.token_logprobs(x, tok, 32))


@pytest.mark.parametrize("V", [200, 9000, 60000])
def test_infinities_and_far_values(V):
    x = rand(8, V, torch.float32, 6)
    x[0, 5] = INF
    x[1, [7, V - 1]] = INF
    x[2] = INF
    x[3] = -INF
    x[3, V // 2] = INF
    x[4] = -3.4e38
    x[5, 3] = 3.4e38
    x[6] *= 1e30
    x[7, ::3] = -2e38
    tok = torch.tensor([5, 8, 0, 1, 2, 3, 4, 3], device="cuda")
    check(x, tok, 12, B.token_logprobs(x, tok, 12))
    p, e, _, _ = B.token_logprobs(x, tok)
    assert p[0] == 0 and p[1] == -INF and p[3] == -INF and e[0] == 0
    assert torch.isfinite(e).all()


def test_confident_rows():
    """Far apart: the log probability of the favourite is -1e-7 and its entropy follows."""
    x = torch.zeros(3, 5000, device="cuda")
    x[0, 17], x[1, 4999], x[2, 0] = 25.0, 40.0, 1000.0
    tok = torch.tensor([17, 4999, 0], device="cuda")
    check(x, tok, 3, B.token_logprobs(x, tok, 3))


def test_tokens_outside_the_vocabulary():
    x = rand(5, 300, torch.float32, 1)
    for dt in (torch.int32, torch.int64):
        tok = torch.tensor([-1, 300, 4, torch.iinfo(dt).min, torch.iinfo(dt).max], dtype=dt, device="cuda")
        p, e, ids, top = B.token_logprobs(x, tok, 2)
        check(x, tok, 2, (p, e, ids, top))
        assert p[0] == 0 and p[1] == 0 and p[2] < 0 and p[3] == 0 and p[4] == 0
    # 64-bit tokens are not cut to 32
    tok = torch.tensor([(1 << 32) + 4] * 5, device="cuda")
    assert (B.token_logprobs(x, tok)[0] == 0).all()


def test_no_rows():
    p, e, ids, top = B.token_logprobs(torch.empty(0, 64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert p.shape == (0,) and e.shape == (0,) and ids.shape == (0, 3) and top.shape == (0, 3)


def test_offsets_past_32_bits():
    """The last rows of logits that take more than 2^31 values (and 2^32 bytes)."""
    V, T = 1 << 20, 2100
    x = torch.zeros(T, V, dtype=torch.float16, device="cuda")
    last = rand(2, V, torch.float16, 3)
    x[T - 2:] = last
    tok = tokens_of(T, V, 1)
    outs = B.token_logprobs(x, tok, 6)
    check(last, tok[T - 2:], 6, [o[T - 2:] for o in outs])


def test_same_result_every_run_streams_and_graphs():
    for T, V, k in ((1, 100000, 20), (300, 9999, 5), (40, 1000, 32)):
        x, tok = rand(T, V, torch.bfloat16, 8), tokens_of(T, V, 8)
        ref = B.token_logprobs(x, tok, k)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            others = [B.token_logprobs(x, tok, k) for _ in range(3)]
        named = B.token_logprobs(x, tok, k, stream=side)
        side.synchronize()
        for o in (*others, named):
            assert all(torch.equal(a, b) for a, b in zip(ref, o))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = B.token_logprobs(x, tok, k)
        x.copy_(rand(T, V, torch.bfloat16, 9))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, B.token_logprobs(x, tok, k)))
        check(x[:4], tok[:4], k, [o[:4] for o in got])
    assert B.status() == F.OK


def test_binding_refuses():
    x, tok = rand(4, 64, torch.float32, 1), tokens_of(4, 64, 1)
    for args, kw in (((x.double(), tok), {}), ((x, tok.float()), {}), ((x, tok[:3]), {}), ((x[0], tok), {}),
                     ((x.t(), tok), {}), ((x, tok.cpu()), {}), ((x, tok.short()), {})):
        with pytest.raises((ValueError, F.MoEError)):
            B.token_logprobs(*args, **kw)
    e = torch.empty(4, device="cuda")
    ids, top = torch.empty(4, 3, dtype=torch.int32, device="cuda"), torch.empty(4, 3, device="cuda")
    for k, out in ((3, (e, e, None, None)), (0, (e, e, ids, top)), (2, (e, e, ids, top)), (3, (e, e, ids.long(), top)),
                   (3, (None, e, ids, top)), (3, (e, e[:2], ids, top)), (3, (e, e, ids.t().contiguous().t(), top))):
        with pytest.raises(ValueError):
            B.token_logprobs(x, tok, k, out=out)
    for k in (33, 65, -1):
        with pytest.raises(F.MoEError):
            B.token_logprobs(x, tok, k)


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V,k", [(310, 66001, 6), (620, 64008, 0)])
def test_long_rows_for_some_rounds_of_ctas(T, V, k, dtype):
    x, tok = rand(T, V, dtype, V + k), tokens_of(T, V, T)
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    outs = B.token_logprobs(x, tok, k)
    check(x[pick], tok[pick], k, tuple(None if o is None else o[pick] for o in outs))
    one = [B.token_logprobs(x[i:i + 1], tok[i:i + 1], k) for i in range(0, T, 37)]   # a row by a cluster
    for j in range(2):
        a, b = torch.cat([o[j] for o in one]), outs[j][::37]
        assert (a - b).abs().max() < 1e-5
    if k:
        assert torch.equal(torch.cat([o[2] for o in one]), outs[2][::37])

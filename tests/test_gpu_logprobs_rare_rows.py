"""token_logprobs on rows that the reading loop cannot settle: few values left by a mask, crowds, and how long they take.

Values against the float64 oracle with the bounds of test_gpu_logprobs; times against ordinary rows of the same sizes,
with bounds a few times what re-reading a row two or three times costs, far below what one element at a time does."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_logprobs import TYPES, check, rand, tokens_of
from tests.test_logprobs_windows import rising
from w4a16_compact_expert_gb300 import block as B
from w4a16_compact_expert_gb300 import moe_w4a16 as F

pytestmark = pytest.mark.gpu


def keep_few(T, V, dtype, keep, seed, mask=-math.inf):
    """Rows with `keep` values at places of their own; the first and the last place of the row among them from 2 on."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, out = rand(T, V, dtype, seed), torch.full((T, V), mask, dtype=dtype, device="cuda")
    for t in range(T):
        at = 1 + torch.randperm(V - 2, device="cuda", generator=g)[:keep]
        if keep > 1:
            at[0], at[1] = 0, V - 1
        out[t, at] = x[t, at]
    return out


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 40003), (3, 5001), (1300, 700)])
@pytest.mark.parametrize("keep", [1, 2, 7, 15, 16, 17, 255, 256, 257, 511, 512, 513, 640])
def test_few_left(T, V, keep, dtype):
    """Around k, and around the number of candidates that a CTA holds."""
    for mask in (-math.inf, torch.finfo(dtype).min):
        x = keep_few(min(T, 40), V, dtype, keep, keep, mask).repeat(-(-T // 40), 1)[:T]
        tok = tokens_of(T, V, 3)
        check(x, tok, 16, B.token_logprobs(x, tok, 16))
    assert B.status() == F.OK


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 66001), (4, 9001), (930, 6003)])
def test_crowds(T, V, dtype):
    """From 500 to 2000 values close together above the others, as many of one value, and a few above those."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for crowd in (500, 512, 513, 700, 2000):
        for near in (False, True):
            x = rand(min(T, 31), V, dtype, crowd, 0.5)
            at = torch.randperm(V, device="cuda", generator=g)[:crowd]
            x[:, at] = 20.0
            if near:
                x[:, at] += (torch.arange(crowd, device="cuda") % 97).to(dtype) / 64
            x[:, at[:5]] = 30.0
            x = x.repeat(-(-T // 31), 1)[:T]
            tok = tokens_of(T, V, 3)
            check(x, tok, 32, B.token_logprobs(x, tok, 32))


def micros(x, tok, k):
    outs = B.token_logprobs(x, tok, k)
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            B.token_logprobs(x, tok, k, out=outs)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 3e-3)
    return sorted(times)[2]


@pytest.mark.parametrize("keep", [1, 19])
def test_few_left_take_a_few_readings(keep):
    """A mask that leaves few tokens: 1000 rows of 131072, 20 best.  Two more readings of a row than an ordinary one; by single
    values and in steps of the CTA they took 20 times as long."""
    T, V = 1000, 131072
    tok = tokens_of(T, V, 1)
    x = rand(T, V, torch.bfloat16, 1)
    few = keep_few(40, V, torch.bfloat16, keep, 2).repeat(T // 40, 1)
    assert micros(few, tok, 20) < 8 * micros(x, tok, 20)


@pytest.mark.parametrize("T,threads", [(930, 128), (500, 512)])
@pytest.mark.parametrize("k", [20, 32])
def test_rows_that_put_too_much_aside(T, threads, k):
    """Values that rise along the row: more windows than there is room for, few values at the last threshold."""
    x = torch.from_numpy(np.stack([rising(threads, i) for i in range(3)])).cuda()
    x = x.repeat(-(-T // 3), 1)[:T]
    tok = tokens_of(T, x.shape[1], 3)
    outs = B.token_logprobs(x, tok, k)
    for at in (slice(0, 4), slice(T - 3, T)):
        check(x[at], tok[at], k, [o[at] for o in outs])


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
def test_the_most_alternatives_take_as_long_as_fewer(dtype):
    """1000 rows of 131072 in no order: read once for 32 alternatives as for 16 (rows read again took 40 times as long)."""
    T, V = 1000, 131072
    tok = tokens_of(T, V, 1)
    x = rand(T, V, dtype, 1)
    assert micros(x, tok, 32) < 2 * micros(x, tok, 16)
    pick = torch.tensor([0, 1, 500, 999], device="cuda")
    check(x[pick], tok[pick], 32, [o[pick] for o in B.token_logprobs(x, tok, 32)])


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 70001), (5, 2000), (610, 129), (1300, 500)])
def test_negative_zero_equals_zero(T, V, dtype):
    """Zeros of either sign where their order decides the ids: the lower index first."""
    k = 16
    rows = []
    x = torch.zeros(T, V, dtype=dtype, device="cuda")
    x[:, 0] = x[:, 5] = -0.0
    rows.append(x)
    x = torch.zeros(T, V, dtype=dtype, device="cuda")
    x[:, ::2] = -0.0
    x[:, 1::9] = -1.0
    rows.append(x.clone())
    x[:, [3, V // 2, V - 1]] = 2.0
    rows.append(x)
    for x in rows:
        signed = x[0].double() - 1e-300 * torch.signbit(x[0]).double()   # an order in which -0 is less
        assert not torch.equal(torch.sort(signed, descending=True, stable=True)[1][:k], torch.sort(x[0].double(), descending=True, stable=True)[1][:k])
        tok = tokens_of(T, V, 1)
        check(x, tok, k, B.token_logprobs(x, tok, k))

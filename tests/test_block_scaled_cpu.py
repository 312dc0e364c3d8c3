"""Block-scaled operators and token log probabilities without a GPU: refusals
of the C entry points (made before anything is enqueued) and pins of the oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from w4a16_compact_expert_gb300 import block as B, build_ext
from w4a16_compact_expert_gb300 import moe_w4a16 as F

P = 0x10000   # a well-aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return B._lib()


def refused(lib, st, word):
    assert st == F.ERR_INVALID_ARG
    assert word in lib.moe_w4a16_last_error(None).decode()


NORM = dict(dtype=0, hidden=64, eps=1e-6, reserved=0, ld_x=0, ld_residual=0, ld_residual_out=0, ld_y=0, ld_q=0)


def norm(lib, T=2, x=P, residual=None, weight=None, residual_out=None, y=P, q=P, q_scale=P, **kw):
    cfg = B.RmsnormConfig(**{**NORM, **kw})
    return lib.moe_w4a16_add_rmsnorm_blocks(ctypes.addressof(cfg), T, x, residual, weight, residual_out, y, q, q_scale, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "dtype"), (dict(hidden=0), "hidden"), (dict(hidden=16385), "hidden"), (dict(eps=math.nan), "eps"),
    (dict(reserved=1), "reserved"), (dict(T=-1), "T"), (dict(ld_q=63), "stride"), (dict(q=None), "together"),
    (dict(q_scale=None), "together"), (dict(q=None, q_scale=None), "required"), (dict(x=None), "NULL"),
    (dict(x=P + 1), "aligned"), (dict(q_scale=P + 2), "aligned")])
def test_norm_refusals(lib, kw, word):
    refused(lib, norm(lib, **kw), word)


LOGPROBS = dict(dtype=2, vocab=64, top_k=4, token_bits=64, ld_logits=0)


def logprobs(lib, T=2, x=P, tokens=P, lp=P, ent=P, ids=P, top=P, **kw):
    cfg = B.LogprobsConfig(**{**LOGPROBS, **kw})
    return lib.moe_w4a16_token_logprobs(ctypes.addressof(cfg), T, x, tokens, lp, ent, ids, top, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 28) + 1), "vocab"),
    (dict(top_k=-1), "top_k"), (dict(top_k=33), "top_k"), (dict(vocab=3), "top_k"), (dict(token_bits=16), "token_bits"),
    (dict(ld_logits=63), "ld_logits"), (dict(T=-1), "T"), (dict(T=(1 << 27) + 1), "T"), (dict(x=None), "NULL"),
    (dict(tokens=None), "NULL"), (dict(lp=None), "NULL"), (dict(ent=None), "NULL"), (dict(ids=None), "go with"),
    (dict(top=None), "go with"), (dict(top_k=0), "go with"), (dict(x=P + 2), "aligned"), (dict(tokens=P + 4), "aligned"),
    (dict(lp=P + 2), "aligned"), (dict(ent=P + 1), "aligned"), (dict(ids=P + 2), "aligned"), (dict(top=P + 2), "aligned")])
def test_logprobs_refusals(lib, kw, word):
    refused(lib, logprobs(lib, **kw), word)


LINEAR = dict(out_dtype=0, n=200, k=256, act=0, reserved=0, reserved2=0, ld_x=0, ld_w=0, ld_x_scale=0, ld_w_scale=0,
              ld_residual=0, ld_out=0)


def linear(lib, T=2, x=P, xs=5 * P, w=2 * P, ws=6 * P, bias=None, res=None, out=3 * P, os=None, **kw):
    cfg = B.LinearBlocksConfig(**{**LINEAR, **kw})
    return lib.moe_w4a16_linear_blocks(ctypes.addressof(cfg), T, x, xs, w, ws, bias, res, out, os, None)


@pytest.mark.parametrize("kw,word", [
    (dict(out_dtype=4), "out_dtype"), (dict(out_dtype=-1), "out_dtype"), (dict(act=6), "activation"),
    (dict(act=-1), "activation"), (dict(reserved=1), "reserved"), (dict(reserved2=1), "reserved"), (dict(n=0), "n outside"),
    (dict(k=0), "n outside"), (dict(n=(1 << 29) + 1), "n outside"), (dict(k=(1 << 24) + 16), "n outside"),
    (dict(T=-1), "T"), (dict(ld_x=255), "stride"), (dict(ld_out=199), "stride"), (dict(ld_residual=1), "stride"),
    (dict(ld_x_scale=1), "stride"), (dict(ld_w_scale=1), "stride"), (dict(k=264), "16 bytes"), (dict(ld_w=264), "16 bytes"),
    (dict(ld_x=1 << 41), "too large"), (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(out=None), "NULL"),
    (dict(xs=None), "NULL"), (dict(ws=None), "NULL"), (dict(os=P), "out_scale"), (dict(out_dtype=3), "out_scale"),
    (dict(out_dtype=3, os=P, res=4 * P), "residual"), (dict(x=P + 8), "aligned"), (dict(w=P + 2), "aligned"),
    (dict(out=P + 1), "aligned"), (dict(res=P + 1), "aligned"), (dict(bias=P + 2), "aligned"), (dict(xs=P + 2), "aligned"),
    (dict(ws=P + 2), "aligned"), (dict(out_dtype=3, os=P + 2), "aligned"), (dict(out=P), "alias"), (dict(out=2 * P), "alias"),
    (dict(out_dtype=3, os=5 * P), "alias"), (dict(out_dtype=3, os=6 * P), "alias")])
def test_linear_refusals(lib, kw, word):
    refused(lib, linear(lib, **kw), word)


def test_null_configs_and_no_rows(lib):
    refused(lib, lib.moe_w4a16_linear_blocks(None, 1, P, P, P, P, None, None, P, None, None), "cfg")
    assert linear(lib, T=0, x=None, xs=None, w=None, ws=None, out=None) == F.OK
    refused(lib, lib.moe_w4a16_add_rmsnorm_blocks(None, 1, P, None, None, None, P, P, P, None), "cfg")
    refused(lib, lib.moe_w4a16_token_logprobs(None, 1, P, P, P, P, P, P, None), "cfg")
    assert norm(lib, T=0, x=None) == F.OK
    assert logprobs(lib, T=0, x=None, tokens=None, lp=None, ent=None, ids=None, top=None) == F.OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        B.token_logprobs(x, torch.zeros(2, dtype=torch.int64), 3)
    with pytest.raises(ValueError, match="CUDA"):
        B.add_rmsnorm(x.half(), quant="blocks")
    with pytest.raises(ValueError, match="quant"):
        B.add_rmsnorm(x.half(), quant="block")


def test_oracle_logprobs_by_hand():
    """p = (1/2, 1/4, 1/4) over the logits (ln 2, 0, 0), and masks."""
    x = np.array([[0.0, math.log(2), 0.0, -math.inf], [math.nan, -math.inf, -math.inf, 5.0], [-math.inf] * 4])
    lp, ent, ids, top, _ = O.token_logprobs(x, np.array([1, 0, 2]), 4)
    assert np.allclose(lp, [math.log(0.5), -math.inf, -math.inf])
    assert np.allclose(ent, [1.5 * math.log(2), 0, 0])
    assert ids.tolist() == [[1, 0, 2, 3], [3, 0, 1, 2], [0, 1, 2, 3]]
    assert np.allclose(top[0], [math.log(0.5), math.log(0.25), math.log(0.25), -math.inf])
    assert top[1, 0] == 0 and (top[1, 1:] == -math.inf).all() and (top[2] == -math.inf).all()


def test_oracle_block_scales_by_hand():
    v = np.zeros((1, 130))
    v[0, 5], v[0, 129] = -448.0, 896.0
    assert O.block_scales(v).tolist() == [[1.0, 2.0]]


def test_oracle_linear_blocks_by_hand():
    """One row of ones: block sums of 128 and 2 times their scales; gate and up blocks of their own."""
    x, w = np.ones((1, 130)), np.ones((2, 130))
    xs = np.array([[2.0, 3.0]])
    out, _, _ = O.linear_blocks(x, w, xs, np.array([[0.5, 10.0]]))
    assert out.tolist() == [[128 * 1.0 + 2 * 30.0] * 2]
    out, pre, _ = O.linear_blocks(x, w, xs, np.array([[0.5, 10.0], [0.25, 0.0]]), act="swiglu")
    assert pre.tolist() == [[188.0, 64.0]] and np.allclose(out, 188.0 * 64.0)


@pytest.mark.parametrize("shape", [(8,), (2, 3, 8)])
def test_norm_in_blocks_refuses_other_dimensions(shape):
    build_ext.build()
    with pytest.raises(ValueError):
        B.add_rmsnorm(torch.zeros(*shape, dtype=torch.float16), quant="blocks")


def test_selftest_of_linear_blocks_refuses(lib):
    def call(T=3, which=0, limit=2000, **kw):
        cfg = B.LinearBlocksConfig(**{**dict(out_dtype=0, n=128, k=1024, act=0), **kw})
        return lib.moe_w4a16_selftest_linear_blocks(ctypes.addressof(cfg), T, P, P, P, P, P, None, which, limit, None)
    refused(lib, call(T=20), "T outside")
    refused(lib, call(T=0), "T outside")
    refused(lib, call(which=3), "which")
    refused(lib, call(limit=10), "limit_cycles")
    refused(lib, call(act=5), "activation")
    refused(lib, call(T=70), "activation")
    refused(lib, call(T=70, act=5, out_dtype=3, which=4), "which")
    assert lib.moe_w4a16_selftest_linear_blocks(None, 3, P, P, P, P, P, None, 0, 2000, None) == F.ERR_INVALID_ARG

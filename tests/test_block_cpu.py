"""Block operators without a GPU: every refusal of the C entry points (made
before anything is enqueued), the binding's checks, and pins of the oracle."""
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


def norm(lib, T=2, x=P, residual=None, weight=None, residual_out=None, y=P, q=None, q_scale=None, **kw):
    cfg = B.RmsnormConfig(**{**NORM, **kw})
    return lib.moe_w4a16_add_rmsnorm(ctypes.addressof(cfg), T, x, residual, weight, residual_out, y, q, q_scale, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=2), "dtype"), (dict(dtype=9), "dtype"), (dict(hidden=0), "hidden"), (dict(hidden=16385), "hidden"),
    (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"), (dict(eps=math.inf), "eps"), (dict(reserved=1), "reserved"),
    (dict(T=-1), "T"), (dict(T=1 << 31), "T"), (dict(ld_x=63), "stride"), (dict(ld_y=-64), "stride"),
    (dict(y=None), "no output"), (dict(q=P), "together"), (dict(q_scale=P), "together"), (dict(x=None), "NULL"),
    (dict(x=P + 1), "aligned"), (dict(residual=P + 1), "aligned"), (dict(weight=P + 1), "aligned"),
    (dict(y=P + 1), "aligned"), (dict(q=P, q_scale=P + 2), "aligned")])
def test_norm_refusals(lib, kw, word):
    refused(lib, norm(lib, **kw), word)


ROUTE = dict(dtype=2, num_experts=64, top_k=8, score=0, num_groups=1, top_groups=1, group_rank=1, renormalize=0,
             scale=1.0, reserved=0, ld_logits=0)


def route(lib, T=2, logits=P, bias=None, ids=P, w=P, **kw):
    cfg = B.RouteConfig(**{**ROUTE, **kw})
    return lib.moe_w4a16_route_scored(ctypes.addressof(cfg), T, logits, bias, ids, w, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "dtype"), (dict(num_experts=0), "num_experts"), (dict(num_experts=513), "num_experts"),
    (dict(score=2), "score"), (dict(num_groups=0), "num_groups"), (dict(num_groups=33), "num_groups"),
    (dict(num_groups=7), "num_groups"), (dict(top_groups=0), "top_groups"), (dict(top_groups=2), "top_groups"),
    (dict(group_rank=0), "group_rank"), (dict(group_rank=3), "group_rank"), (dict(top_k=0), "top_k"),
    (dict(top_k=33), "top_k"), (dict(num_groups=16, top_groups=1, top_k=5), "top_k"),
    (dict(num_experts=4), "top_k"), (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"),
    (dict(reserved=2), "reserved"), (dict(ld_logits=63), "ld_logits"), (dict(T=-1), "T"), (dict(logits=None), "NULL"),
    (dict(ids=None), "NULL"), (dict(w=None), "NULL"), (dict(logits=P + 2), "aligned"), (dict(bias=P + 2), "aligned"),
    (dict(ids=P + 2), "aligned"), (dict(w=P + 1), "aligned")])
def test_route_refusals(lib, kw, word):
    refused(lib, route(lib, **kw), word)


LINEAR = dict(in_dtype=0, out_dtype=0, n=64, k=64, act=0, reserved=0, ld_x=0, ld_w=0, ld_residual=0, ld_out=0)


def linear(lib, T=2, x=P, w=2 * P, xs=None, ws=None, bias=None, res=None, out=3 * P, **kw):
    cfg = B.LinearConfig(**{**LINEAR, **kw})
    return lib.moe_w4a16_linear(ctypes.addressof(cfg), T, x, w, xs, ws, bias, res, out, None)


@pytest.mark.parametrize("kw,word", [
    (dict(in_dtype=2), "in_dtype"), (dict(out_dtype=3), "out_dtype"), (dict(act=6), "activation"),
    (dict(act=-1), "activation"), (dict(reserved=1), "reserved"), (dict(n=0), "n outside"), (dict(k=0), "n outside"),
    (dict(n=(1 << 29) + 1), "n outside"), (dict(k=(1 << 24) + 8), "n outside"),
    (dict(T=-1), "T"), (dict(ld_x=63), "stride"), (dict(ld_out=63), "stride"), (dict(ld_residual=1), "stride"),
    (dict(k=60), "16 bytes"), (dict(ld_w=68), "16 bytes"), (dict(in_dtype=3, k=72, xs=P, ws=P), "16 bytes"),
    (dict(ld_x=1 << 40), "too large"), (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(out=None), "NULL"),
    (dict(in_dtype=3), "x_scale"), (dict(in_dtype=3, xs=P), "x_scale"), (dict(xs=P), "x_scale"), (dict(ws=P), "x_scale"),
    (dict(x=P + 8), "aligned"), (dict(w=P + 2), "aligned"), (dict(out=P + 1), "aligned"), (dict(res=P + 1), "aligned"),
    (dict(bias=P + 2), "aligned"), (dict(out=P), "alias"), (dict(out=2 * P), "alias")])
def test_linear_refusals(lib, kw, word):
    refused(lib, linear(lib, **kw), word)


def test_null_configs_and_no_rows(lib):
    refused(lib, lib.moe_w4a16_add_rmsnorm(None, 1, P, None, None, None, P, None, None, None), "cfg")
    refused(lib, lib.moe_w4a16_route_scored(None, 1, P, None, P, P, None), "cfg")
    refused(lib, lib.moe_w4a16_linear(None, 1, P, P, None, None, None, None, P, None), "cfg")
    assert norm(lib, T=0, x=None) == F.OK
    assert route(lib, T=0, logits=None, ids=None, w=None) == F.OK
    assert linear(lib, T=0, x=None, w=None, out=None) == F.OK


def test_routed_forward_without_a_handle(lib):
    assert lib.moe_w4a16_forward_routed(None, P, 1, P, P, 0, P, None) == F.ERR_INVALID_ARG


def test_routed_forward_refuses_host_tensors():
    m = object.__new__(F.MoELayer)   # refused before the library is called
    m.h, m.cfg = None, F.Config(hidden=64, inter=64, num_experts=4, top_k=2)
    x, ids, w = torch.zeros(3, 64, dtype=torch.float16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="CUDA device"):
        m.forward_routed(x, ids, w)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(2, 64, dtype=torch.float16)
    for f in (lambda: B.add_rmsnorm(x), lambda: B.linear(x, x), lambda: B.route_scored(x, 2)):
        with pytest.raises(ValueError):   # host tensors
            f()


def test_oracle_norm_by_hand():
    s, n = O.add_rmsnorm(np.array([[3.0, 0.0]]), np.array([[0.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert s.tolist() == [[3.0, 4.0]]
    assert np.allclose(n, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]], rtol=1e-15)


def test_oracle_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    ids, w = O.route_scored(l, None, 2)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[0.4, 0.3]])
    ids, w = O.route_scored(l, np.array([1.0, 0, 0, 0]), 2, renormalize=True, scale=2.0)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[0.4, 1.6]])
    ids, w = O.route_scored(l, None, 2, groups=2, top_groups=1, group_rank=2, score="sigmoid")
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[0.8, 0.75]])
    ids, w = O.route_scored(np.array([[-np.inf, 0.0, np.nan]]), None, 2, renormalize=True)
    assert ids.tolist() == [[1, 0]] and w.tolist() == [[1.0, 0.0]]
    # group 0's two smaller choices together beat group 1's single largest
    ids, _ = O.route_scored(np.log(np.array([[3.0, 3.0, 4.0, 0.5]])), None, 1, groups=2, top_groups=1, group_rank=2)
    assert ids.tolist() == [[0]]


def test_oracle_linear_by_hand():
    x, w = np.array([[1.0, 2.0]]), np.array([[1.0, 1.0], [0.0, -1.0]])
    out, pre, mag = O.linear(x, w, bias=np.array([0.0, 1.0]), act="relu", residual=np.array([[10.0, 20.0]]))
    assert out.tolist() == [[13.0, 20.0]] and pre.tolist() == [[3.0, -1.0]] and mag.tolist() == [[3.0, 2.0]]
    out, *_ = O.linear(x, w, act="swiglu")
    assert np.allclose(out, [[-2 * 3 / (1 + math.exp(-3))]])
    out, *_ = O.linear(x, w, x_scale=np.array([2.0]), w_scale=np.array([1.0, 3.0]))
    assert out.tolist() == [[6.0, -12.0]]


def test_no_copy_is_shared_over_a_cluster():
    """Every copy loads into one CTA: the library also runs as one of several replicas on a machine, on any device memory."""
    import glob
    import os
    import re
    sources = [f for e in ("cu", "cuh", "h", "cpp") for f in glob.glob(os.path.join(build_ext.CSRC, "*." + e))]
    assert len(sources) > 10
    for path in sources:
        with open(path) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())   # joined string literals
        for stmt in re.findall(r"cp\.async\.bulk[^;]*", text):
            assert "multi" + "cast" not in stmt, (os.path.basename(path), stmt)


@pytest.mark.parametrize("kw,word", [
    (dict(in_dtype=1), "F16"), (dict(out_dtype=2), "F16"), (dict(act=1), "F16"), (dict(T=0), "T outside"),
    (dict(T=17), "T outside"), (dict(T=64), "T outside"), (dict(which=-1), "which"), (dict(which=3), "which"),
    (dict(limit=999), "limit"), (dict(limit=(1 << 31) + 1), "limit"), (dict(k=0), "n outside"), (dict(x=None), "NULL"),
    (dict(w=P + 2), "aligned")])
def test_linear_selftest_refusals(lib, kw, word):
    a = dict(T=2, x=P, w=2 * P, which=0, limit=10_000)
    cfg = B.LinearConfig(**{**LINEAR, **{k: v for k, v in kw.items() if k not in a}})
    a.update({k: v for k, v in kw.items() if k in a})
    refused(lib, lib.moe_w4a16_selftest_linear(ctypes.addressof(cfg), a["T"], a["x"], a["w"], 3 * P, a["which"],
                                               a["limit"], None), word)


def test_routed_forward_takes_the_stream_of_the_layers_device(monkeypatch):
    class OnDevice:   # what forward_routed looks at of a CUDA tensor
        def __init__(self, t):
            self.dtype, self.shape, self.device, self.dim = t.dtype, t.shape, "cuda:1", t.dim

        def get_device(self):
            return 1

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return P

    class Stream:
        def __init__(self, device):
            self.cuda_stream = 1000 + (0 if device is None else device)

    calls = []

    class Lib:
        def moe_w4a16_forward_routed(self, *a):
            calls.append(a)
            return F.OK

        def moe_w4a16_destroy(self, h):
            pass

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(device))
    m = object.__new__(F.MoELayer)
    m.h, m.lib, m.cfg = None, Lib(), F.Config(hidden=64, inter=64, num_experts=4, top_k=2, device=1)
    x = OnDevice(torch.zeros(3, 64, dtype=torch.float16))
    m.forward_routed(x, OnDevice(torch.zeros(3, 2, dtype=torch.int32)), OnDevice(torch.zeros(3, 2)), out=x)
    assert calls[0][-1] == 1001


def test_another_torch_rebuilds_the_binding(monkeypatch):
    build_ext.build()
    assert build_ext.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build_ext.up_to_date()

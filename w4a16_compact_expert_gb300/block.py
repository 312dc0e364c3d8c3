"""Block operators: what an MoE block needs around its routed experts.

  add_rmsnorm   residual addition + root-mean-square norm (+ an 8-bit copy)
  linear        matrix product with scales, bias, activation and residual
  route_scored  expert ids and weights from router logits

The definitions, limits and masking rules are those of moe_w4a16_add_rmsnorm,
moe_w4a16_linear and moe_w4a16_route_scored in include/moe_w4a16.h; this
module and the compiled _block beside it check tensors and marshal pointers.
Inputs are CUDA tensors of one device; a wrong shape, type or layout raises
ValueError, an error of the library MoEError.  Rows may be strided (the last
dimension contiguous).  There is no backward pass: outputs carry no gradient.
Outputs are allocated unless given; with stream=None work goes to the
current stream.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os

import torch

from . import moe_w4a16 as _m

_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}
_F32, _I32, _E4M3 = torch.float32, torch.int32, torch.float8_e4m3fn


class RmsnormConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("hidden", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("ld_x", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_residual_out", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_q", ctypes.c_int64)]


class RouteConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_rank", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("ld_logits", ctypes.c_int64)]


class LinearConfig(ctypes.Structure):
    _fields_ = [("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("act", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("ld_x", ctypes.c_int64), ("ld_w", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_out", ctypes.c_int64)]


@functools.lru_cache(maxsize=None)
def _lib():
    lib = _m.load_library()
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.moe_w4a16_add_rmsnorm.argtypes = [vp, i64] + [vp] * 8
    lib.moe_w4a16_route_scored.argtypes = [vp, i64] + [vp] * 5
    lib.moe_w4a16_linear.argtypes = [vp, i64] + [vp] * 8
    lib.moe_w4a16_block_status.argtypes = []
    lib.moe_w4a16_selftest_linear.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int32, i64, vp]
    return lib


_native = None   # the compiled module _block


def _load():
    global _native
    _lib()
    path = os.path.join(os.path.dirname(_m.LIB_PATH), "_block.so")
    if not os.path.exists(path):
        raise RuntimeError(f"binding not built: {path} (run __graft_entry__.build())")
    spec = importlib.util.spec_from_file_location("_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.set_error(_m.MoEError)
    _native = mod
    return mod


def _empty(shape, dtype, like, stream):
    """An output, allocated for the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def add_rmsnorm(x, residual=None, weight=None, *, eps: float = 1e-6, norm: bool = True, quant: bool = False, out=None,
                stream=None):
    """s = x + residual, n = s / sqrt(mean s^2 + eps) * weight, per row of x [T, H] (fp16 or bf16).

    Returns (y, s, q, q_scale): y = n in x's type (None with norm=False), s in
    x's type (None without a residual), q = n / q_scale in E4M3 with one FP32
    scale per row (both None unless quant).  out: the same four, to be
    written (None where not returned); s may be x or residual, y may be x."""
    if out is None:
        dt = x.dtype
        y = _empty(x.shape, dt, x, stream) if norm else None
        s = _empty(x.shape, dt, x, stream) if residual is not None else None
        q = _empty(x.shape, _E4M3, x, stream) if quant else None
        qs = _empty(x.shape[:1], _F32, x, stream) if quant else None
    else:
        y, s, q, qs = out
        if (y is None) == norm or (s is None) != (residual is None) or (q is None) == quant or (qs is None) == quant:
            raise ValueError("out must hold (y, s, q, q_scale), None exactly where nothing is returned")
    (_native or _load()).add_rmsnorm(x, residual, weight, eps, y, s, q, qs, stream)
    return y, s, q, qs


def route_scored(logits, top_k: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renormalize: bool = False, scale: float = 1.0, out=None, stream=None):
    """Expert ids [T, k] int32 and weights [T, k] fp32 from logits [T, E] (fp32, fp16 or bf16).

    score "softmax" or "sigmoid"; bias [E] fp32 is added to the scores for the
    selection only; of `groups` equal groups of experts the `top_groups` with
    the largest sum of their `group_rank` (1 or 2) largest choices stay
    eligible; the weights are the scores of the chosen, divided by their sum
    if renormalize, times scale.  out: (ids, weights) to be written."""
    code = _SCORES.get(score)
    if code is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if out is None:
        shape = (logits.shape[0], top_k)
        ids, w = _empty(shape, _I32, logits, stream), _empty(shape, _F32, logits, stream)
    else:
        ids, w = out
    (_native or _load()).route_scored(logits, bias, ids, w, top_k, code, groups, top_groups, group_rank, renormalize,
                                      scale, stream)
    return ids, w


def linear(x, w, *, bias=None, act: str = "none", residual=None, x_scale=None, w_scale=None, out_dtype=None, out=None,
           stream=None):
    """act(x_scale w_scale x w^T + bias) + residual for x [T, K] and w [N, K] (fp16, bf16, or E4M3 with FP32
    scales per row of x and of w); bias fp32.

    act: none, relu, gelu, gelu_tanh, silu, or swiglu (w holds N gate rows,
    then N up rows; silu(gate) * up).  The output [T, N] has out_dtype (x's
    type; fp16 for E4M3), fp16, bf16 or fp32, like the residual; it may be
    the residual."""
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of " + ", ".join(_ACTS))
    if out is None:
        n = w.shape[0] // 2 if code == 5 else w.shape[0]
        out = _empty((x.shape[0], n), out_dtype or (torch.float16 if x.dtype is _E4M3 else x.dtype), x, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    (_native or _load()).linear(x, w, x_scale, w_scale, bias, residual, out, code, stream)
    return out


def status() -> int:
    """Synchronises and clears the status of the block operators: OK or ERR_TIMEOUT."""
    return _lib().moe_w4a16_block_status()


def selftest_timeout(x, w, which: int, limit_cycles: int) -> None:
    """Enqueue linear(x, w) with warps that stop early (see moe_w4a16_selftest_linear); x [T, K] and w [N, K] fp16."""
    (T, K), N = x.shape, w.shape[0]
    out = torch.empty(T, N, dtype=torch.float16, device=x.device)
    cfg = LinearConfig(n=N, k=K)   # F16 in and out, no activation
    lib = _lib()
    st = lib.moe_w4a16_selftest_linear(ctypes.addressof(cfg), T, _m._ptr(x), _m._ptr(w), _m._ptr(out), int(which),
                                       int(limit_cycles), _m._stream(None))
    if st != _m.OK:
        raise _m.MoEError(st, lib.moe_w4a16_last_error(None).decode())


class MoEBlock:
    """The feed-forward half of a decoder block around one MoELayer:

        s   = x + residual                       the residual stream
        n   = rmsnorm(s) * norm_weight           (and n in E4M3 for an 8-bit shared expert)
        ids, w = route_scored(n router_w^T)
        out = sum_j w_j expert_ids_j(n) + shared(n),   shared(n) = down(silu(gate n) * (up n))

    Returns (out, s); the next block adds them up.  layer: a MoELayer with
    experts and slot table set.  router_w fp16 [E, H]; shared: None or
    (gate_up, down) with gate_up [2 Is, H] in fp16, or in E4M3 with
    shared_scale fp32 [2 Is], and down fp16 [H, Is].  route: the keyword
    arguments of route_scored.  The layer's rule on streams (one stream per
    handle, or ordered by events) is the block's."""

    def __init__(self, layer, norm_weight, router_w, shared=None, shared_scale=None, eps: float = 1e-6, **route):
        self.layer, self.norm_weight, self.router_w, self.eps, self.route = layer, norm_weight, router_w, eps, route
        self.gate_up, self.down = shared if shared is not None else (None, None)
        self.scale = shared_scale
        self.quant = self.gate_up is not None and self.gate_up.dtype is _E4M3
        if self.quant != (shared_scale is not None):
            raise ValueError("shared_scale goes with an E4M3 gate_up")

    def __call__(self, x, residual=None, stream=None):
        n, s, q, qs = add_rmsnorm(x, residual, self.norm_weight, eps=self.eps, quant=self.quant, stream=stream)
        logits = linear(n, self.router_w, out_dtype=_F32, stream=stream)
        ids, w = route_scored(logits, self.layer.cfg.top_k, stream=stream, **self.route)
        out = _empty(n.shape, n.dtype, n, stream)
        self.layer.forward_routed(n, ids, w, out=out, stream=stream)
        if self.gate_up is not None:
            h = linear(q if self.quant else n, self.gate_up, act="swiglu", x_scale=qs, w_scale=self.scale, stream=stream)
            linear(h, self.down, residual=out, out=out, stream=stream)
        return out, x if s is None else s

"""Block operators: what an MoE block needs around its routed experts.

  add_rmsnorm   residual addition + root-mean-square norm (+ an 8-bit copy)
  linear        matrix product with scales, bias, activation and residual
  linear_blocks the same of E4M3 operands with a scale per block of 128
  route_scored  expert ids and weights from router logits
  token_logprobs  log probabilities of given tokens, entropies, best alternatives

The definitions, limits and masking rules are those of the functions of the
same names (moe_w4a16_...) in include/moe_w4a16.h; this module and the
compiled _block beside it check tensors and marshal pointers.
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
BLOCK = 128   # values that share a scale in the block-scaled operators
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


class LinearBlocksConfig(ctypes.Structure):
    _fields_ = [("out_dtype", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("reserved2", ctypes.c_int32), ("ld_x", ctypes.c_int64),
                ("ld_w", ctypes.c_int64), ("ld_x_scale", ctypes.c_int64), ("ld_w_scale", ctypes.c_int64),
                ("ld_residual", ctypes.c_int64), ("ld_out", ctypes.c_int64)]


class LogprobsConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("vocab", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("token_bits", ctypes.c_int32), ("ld_logits", ctypes.c_int64)]


@functools.lru_cache(maxsize=None)
def _lib():
    lib = _m.load_library()
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.moe_w4a16_add_rmsnorm.argtypes = [vp, i64] + [vp] * 8
    lib.moe_w4a16_route_scored.argtypes = [vp, i64] + [vp] * 5
    lib.moe_w4a16_linear.argtypes = [vp, i64] + [vp] * 8
    lib.moe_w4a16_add_rmsnorm_blocks.argtypes = [vp, i64] + [vp] * 8
    lib.moe_w4a16_linear_blocks.argtypes = [vp, i64] + [vp] * 9
    lib.moe_w4a16_token_logprobs.argtypes = [vp, i64] + [vp] * 7
    lib.moe_w4a16_block_status.argtypes = []
    lib.moe_w4a16_selftest_linear.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int32, i64, vp]
    lib.moe_w4a16_selftest_linear_blocks.argtypes = [vp, i64] + [vp] * 6 + [ctypes.c_int32, i64, vp]
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


def _blocks(n):
    return -(-n // BLOCK)


def _empty_rows8(T, n, like, stream):
    """An E4M3 [T, n] whose rows start on the 16-byte grid, as the next linear_blocks wants its x."""
    pad = -n % 16
    return _empty((T, n + pad), _E4M3, like, stream)[:, :n] if pad else _empty((T, n), _E4M3, like, stream)


def add_rmsnorm(x, residual=None, weight=None, *, eps: float = 1e-6, norm: bool = True, quant=False, out=None,
                stream=None):
    """s = x + residual, n = s / sqrt(mean s^2 + eps) * weight, per row of x [T, H] (fp16 or bf16).

    Returns (y, s, q, q_scale): y = n in x's type (None with norm=False), s in
    x's type (None without a residual), q = n / q_scale in E4M3 with one FP32
    scale per row (both None unless quant).  quant="blocks": a scale per row
    and 128 values instead, q_scale [T, ceil(H / 128)], as linear_blocks takes
    them (rows allocated on the 16-byte grid).  out: the same four, to be written (None where not returned); s may
    be x or residual, y may be x."""
    blocks = False
    if quant is not False and quant is not True:   # the smallest calls are bound by the host
        blocks = quant == "blocks"
        if not blocks and isinstance(quant, str):
            raise ValueError("quant must be True, False or 'blocks'")
        quant = bool(quant)
    if out is None:
        dt = x.dtype
        y = _empty(x.shape, dt, x, stream) if norm else None
        s = _empty(x.shape, dt, x, stream) if residual is not None else None
        rows = blocks and x.dim() == 2   # else refused below
        q = (_empty_rows8(*x.shape, x, stream) if rows else _empty(x.shape, _E4M3, x, stream)) if quant else None
        qs = _empty((x.shape[0], _blocks(x.shape[1])) if rows else x.shape[:1], _F32, x, stream) if quant else None
    else:
        y, s, q, qs = out
        if (y is None) == norm or (s is None) != (residual is None) or (q is None) == quant or (qs is None) == quant:
            raise ValueError("out must hold (y, s, q, q_scale), None exactly where nothing is returned")
    (_native or _load()).add_rmsnorm(x, residual, weight, eps, y, s, q, qs, stream, blocks)
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


def linear_blocks(x, w, x_scale, w_scale, *, bias=None, act: str = "none", residual=None, out_dtype=None, out=None,
                  out_scale=None, stream=None):
    """act(x w^T + bias) + residual for E4M3 x [T, K] with fp32 x_scale [T, ceil(K / 128)] and E4M3 w [N, K] with
    fp32 w_scale [ceil(N / 128), ceil(K / 128)], a scale per 128 x 128 block; bias fp32.

    act as in linear; for swiglu w holds N gate rows, then N up rows, and
    w_scale the blocks of the gate, then those of the up rows.  The output
    [T, N] has out_dtype (fp16 unless given), fp16, bf16, fp32 like the
    residual, which it may be, or float8_e4m3fn: then it is returned with its
    scales [T, ceil(N / 128)] as (out, out_scale), fit to be another call's x
    and x_scale (rows that are allocated here start on the 16-byte grid)."""
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of " + ", ".join(_ACTS))
    if out is None:
        n = w.shape[0] // 2 if code == 5 else w.shape[0]
        out = (_empty_rows8(x.shape[0], n, x, stream) if out_dtype is _E4M3 else
               _empty((x.shape[0], n), out_dtype or torch.float16, x, stream))
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    quant = out.dtype is _E4M3
    if quant and out_scale is None:
        out_scale = _empty((out.shape[0], _blocks(out.shape[-1])), _F32, x, stream)
    (_native or _load()).linear_blocks(x, w, x_scale, w_scale, bias, residual, out, out_scale, code, stream)
    return (out, out_scale) if quant else out


def token_logprobs(logits, tokens, top_k: int = 0, *, out=None, stream=None):
    """(logprob [T], entropy [T], top_ids [T, k] int32, top_logprobs [T, k]), fp32, of the softmax of logits [T, V]
    (fp32, fp16 or bf16).

    logprob is ln p of tokens [T] (int32 or int64; 0 for a token outside the
    vocabulary, as padding has), entropy in nats; top_ids and top_logprobs, None
    for top_k = 0, the k most likely tokens, largest first, ties to the lower
    id.  Logits of -inf or NaN are masked.  out: the same four, to be written."""
    if out is None:
        T = logits.shape[0]
        p, e = _empty((T,), _F32, logits, stream), _empty((T,), _F32, logits, stream)
        ids = _empty((T, top_k), _I32, logits, stream) if top_k > 0 else None
        top = _empty((T, top_k), _F32, logits, stream) if top_k > 0 else None
    else:
        p, e, ids, top = out
        if p is None or e is None or (ids is None) != (top_k == 0) or (top is None) != (top_k == 0):
            raise ValueError("out must hold (logprob, entropy, top_ids, top_logprobs), None exactly where nothing is returned")
    (_native or _load()).token_logprobs(logits, tokens, p, e, ids, top, top_k, stream)
    return p, e, ids, top


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


def selftest_blocks_timeout(x, w, x_scale, w_scale, which: int, limit_cycles: int) -> None:
    """The same of linear_blocks (see moe_w4a16_selftest_linear_blocks): up to 16 tokens fp16 out, above 64 swiglu to E4M3."""
    (T, K), wide = x.shape, x.shape[0] > 64
    N = w.shape[0] // 2 if wide else w.shape[0]
    out = torch.empty(T, N, dtype=_E4M3 if wide else torch.float16, device=x.device)
    out_scale = torch.empty(T, _blocks(N), dtype=_F32, device=x.device) if wide else None
    cfg = LinearBlocksConfig(out_dtype=3 if wide else 0, n=N, k=K, act=_ACTS["swiglu" if wide else "none"])
    lib = _lib()
    st = lib.moe_w4a16_selftest_linear_blocks(ctypes.addressof(cfg), T, _m._ptr(x), _m._ptr(x_scale), _m._ptr(w),
                                              _m._ptr(w_scale), _m._ptr(out), _m._ptr(out_scale), int(which),
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
    shared_scale fp32 [2 Is], and down fp16 [H, Is].  Or both in E4M3 with a
    scale per 128 x 128 block: shared_scale = (that of gate_up, that of down) as
    linear_blocks takes them; the norm and the gated product then write E4M3
    with a scale per 128 values.  route: the keyword arguments of route_scored.
    The layer's rule on streams (one stream per handle, or ordered by events)
    is the block's."""

    def __init__(self, layer, norm_weight, router_w, shared=None, shared_scale=None, eps: float = 1e-6, **route):
        self.layer, self.norm_weight, self.router_w, self.eps, self.route = layer, norm_weight, router_w, eps, route
        self.gate_up, self.down = shared if shared is not None else (None, None)
        self.scale = shared_scale
        self.blocks = isinstance(shared_scale, (tuple, list))
        self.quant = self.gate_up is not None and self.gate_up.dtype is _E4M3
        if self.quant != (shared_scale is not None):
            raise ValueError("shared_scale goes with an E4M3 gate_up")
        if self.blocks:
            if len(shared_scale) != 2:
                raise ValueError("shared_scale in blocks is a pair, of gate_up and of down")
            self.quant = "blocks"

    def __call__(self, x, residual=None, stream=None):
        n, s, q, qs = add_rmsnorm(x, residual, self.norm_weight, eps=self.eps, quant=self.quant, stream=stream)
        logits = linear(n, self.router_w, out_dtype=_F32, stream=stream)
        ids, w = route_scored(logits, self.layer.cfg.top_k, stream=stream, **self.route)
        out = _empty(n.shape, n.dtype, n, stream)
        self.layer.forward_routed(n, ids, w, out=out, stream=stream)
        if self.blocks:
            h, hs = linear_blocks(q, self.gate_up, qs, self.scale[0], act="swiglu", out_dtype=_E4M3, stream=stream)
            linear_blocks(h, self.down, hs, self.scale[1], residual=out, out=out, stream=stream)
        elif self.gate_up is not None:
            h = linear(q if self.quant else n, self.gate_up, act="swiglu", x_scale=qs, w_scale=self.scale, stream=stream)
            linear(h, self.down, residual=out, out=out, stream=stream)
        return out, x if s is None else s

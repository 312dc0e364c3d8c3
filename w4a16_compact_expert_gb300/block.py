"""Block operators: what an MoE block needs around its routed experts.

  add_rmsnorm   residual addition + root-mean-square norm (+ an 8-bit copy)
  linear        matrix product with scales, bias, activation and residual
  route_scored  expert ids and weights from router logits

The definitions, limits and masking rules are those of moe_w4a16_add_rmsnorm,
moe_w4a16_linear and moe_w4a16_route_scored in include/moe_w4a16.h; this
module checks tensors and marshals pointers.  Inputs are CUDA tensors of one
device; a wrong shape, type or layout raises ValueError, an error of the
library MoEError.  Rows may be strided (the last dimension contiguous).
Outputs are allocated unless given; with stream=None work goes to the
current stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import moe_w4a16 as _m

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.float8_e4m3fn: 3}
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
    return lib


# A config is plain numbers (shapes, types, strides): kept once per combination.
@functools.lru_cache(maxsize=4096)
def _config(cls, *fields):
    cfg = cls(*fields)
    return cfg, ctypes.addressof(cfg)


def _call(fn, stream, device, *args):
    """fn(*args, stream) with `device` current."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(*args, _m._stream(stream))
    else:
        st = fn(*args, torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream)
    if st != _m.OK:
        raise _m.MoEError(st, _lib().moe_w4a16_last_error(None).decode())


def _empty(shape, dtype, like, stream):
    """An output, allocated for the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rows(name, t, T, n, dtype, device):
    """Checks a [T, n] tensor with contiguous rows; returns (pointer, row stride)."""
    if t.dtype != dtype or t.get_device() != device or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor on the device of the other arguments")
    if t.shape[0] != T or t.shape[1] != n:
        raise ValueError(f"{name} must have shape ({T}, {n}), got {tuple(t.shape)}")
    ld, inner = t.stride()
    if (inner != 1 and n > 1) or (ld < n and T > 1):
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld if ld >= n else n


def _vector(name, t, n, dtype, device):
    if t.dtype != dtype or t.get_device() != device or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on the device of the other arguments")
    return t.data_ptr()


def _input(name, x, dtypes):
    if x.dtype not in dtypes or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    return x.get_device()


_NORM_TYPES = (torch.float16, torch.bfloat16)
_LOGIT_TYPES = (torch.float32, torch.float16, torch.bfloat16)
_LINEAR_TYPES = (torch.float16, torch.bfloat16, torch.float8_e4m3fn)


def add_rmsnorm(x, residual=None, weight=None, *, eps: float = 1e-6, norm: bool = True, quant: bool = False, out=None,
                stream=None):
    """s = x + residual, n = s / sqrt(mean s^2 + eps) * weight, per row of x [T, H] (fp16 or bf16).

    Returns (y, s, q, q_scale): y = n in x's type (None with norm=False), s in
    x's type (None without a residual), q = n / q_scale in E4M3 with one FP32
    scale per row (both None unless quant).  out: the same four, to be
    written (None where not returned); s may be x or residual, y may be x."""
    dev = _input("x", x, _NORM_TYPES)
    T, H = x.shape
    dt = x.dtype
    px, ldx = _rows("x", x, T, H, dt, dev)
    pr = ldr = pso = ldso = py = ldy = pq = ldq = pqs = pw = 0
    if out is None:
        y = _empty((T, H), dt, x, stream) if norm else None
        s = _empty((T, H), dt, x, stream) if residual is not None else None
        q = _empty((T, H), _E4M3, x, stream) if quant else None
        qs = _empty((T,), _F32, x, stream) if quant else None
    else:
        y, s, q, qs = out
        if (y is None) == norm or (s is None) != (residual is None) or (q is None) == quant or (qs is None) == quant:
            raise ValueError("out must hold (y, s, q, q_scale), None exactly where nothing is returned")
    if residual is not None:
        pr, ldr = _rows("residual", residual, T, H, dt, dev)
        pso, ldso = _rows("out s", s, T, H, dt, dev)
    if weight is not None:
        pw = _vector("weight", weight, H, dt, dev)
    if norm:
        py, ldy = _rows("out y", y, T, H, dt, dev)
    if quant:
        pq, ldq = _rows("out q", q, T, H, _E4M3, dev)
        pqs = _vector("out q_scale", qs, T, _F32, dev)
    cfg = _config(RmsnormConfig, _DTYPES[dt], H, eps, 0, ldx, ldr, ldso, ldy, ldq)[1]
    _call(_lib().moe_w4a16_add_rmsnorm, stream, dev, cfg, T, px, pr, pw, pso, py, pq, pqs)
    return y, s, q, qs


def route_scored(logits, top_k: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renormalize: bool = False, scale: float = 1.0, out=None, stream=None):
    """Expert ids [T, k] int32 and weights [T, k] fp32 from logits [T, E] (fp32, fp16 or bf16).

    score "softmax" or "sigmoid"; bias [E] fp32 is added to the scores for the
    selection only; of `groups` equal groups of experts the `top_groups` with
    the largest sum of their `group_rank` (1 or 2) largest choices stay
    eligible; the weights are the scores of the chosen, divided by their sum
    if renormalize, times scale.  out: (ids, weights) to be written."""
    dev = _input("logits", logits, _LOGIT_TYPES)
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    pl, ld = _rows("logits", logits, T, E, logits.dtype, dev)
    if out is None:
        ids, w = _empty((T, top_k), _I32, logits, stream), _empty((T, top_k), _F32, logits, stream)
    else:
        ids, w = out
    for name, t, d in (("out ids", ids, _I32), ("out weights", w, _F32)):
        if _rows(name, t, T, top_k, d, dev)[1] != top_k:
            raise ValueError(f"{name} must be contiguous")
    pb = _vector("bias", bias, E, _F32, dev) if bias is not None else 0
    cfg = _config(RouteConfig, _DTYPES[logits.dtype], E, top_k, _SCORES[score], groups, top_groups, group_rank,
                  int(bool(renormalize)), scale, 0, ld)[1]
    _call(_lib().moe_w4a16_route_scored, stream, dev, cfg, T, pl, pb, ids.data_ptr(), w.data_ptr())
    return ids, w


def linear(x, w, *, bias=None, act: str = "none", residual=None, x_scale=None, w_scale=None, out_dtype=None, out=None,
           stream=None):
    """act(x_scale w_scale x w^T + bias) + residual for x [T, K] and w [N, K] (fp16, bf16, or E4M3 with FP32
    scales per row of x and of w); bias fp32.

    act: none, relu, gelu, gelu_tanh, silu, or swiglu (w holds N gate rows,
    then N up rows; silu(gate) * up).  The output [T, N] has out_dtype (x's
    type; fp16 for E4M3), fp16, bf16 or fp32, like the residual; it may be
    the residual."""
    dev = _input("x", x, _LINEAR_TYPES)
    T, K = x.shape
    dt = x.dtype
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of " + ", ".join(_ACTS))
    M = w.shape[0]
    if code == 5 and M % 2:
        raise ValueError("swiglu needs an even number of rows in w")
    N = M // 2 if code == 5 else M
    px, ldx = _rows("x", x, T, K, dt, dev)
    pw, ldw = _rows("w", w, M, K, dt, dev)
    if out is None:
        out = _empty((T, N), out_dtype or (torch.float16 if dt is _E4M3 else dt), x, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    ot = out.dtype
    if ot not in _LOGIT_TYPES:
        raise ValueError("the output must be fp16, bf16 or fp32")
    po, ldo = _rows("out", out, T, N, ot, dev)
    pb = _vector("bias", bias, M, _F32, dev) if bias is not None else 0
    pr = ldr = pxs = pws = 0
    if residual is not None:
        pr, ldr = _rows("residual", residual, T, N, ot, dev)
    if dt is _E4M3:
        if x_scale is None or w_scale is None:
            raise ValueError("E4M3 needs x_scale and w_scale")
        pxs, pws = _vector("x_scale", x_scale, T, _F32, dev), _vector("w_scale", w_scale, M, _F32, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale go with E4M3 only")
    cfg = _config(LinearConfig, _DTYPES[dt], _DTYPES[ot], N, K, code, 0, ldx, ldw, ldr, ldo)[1]
    _call(_lib().moe_w4a16_linear, stream, dev, cfg, T, px, pw, pxs, pws, pb, pr, po)
    return out


def status() -> int:
    """Synchronises and clears the status of the block operators: OK or ERR_TIMEOUT."""
    return _lib().moe_w4a16_block_status()

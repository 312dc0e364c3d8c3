"""Float64 numpy oracle of the block operators (test infrastructure; shares
no code with the CUDA path): the definitions of include/moe_w4a16.h, row by row."""
from __future__ import annotations

import math

import numpy as np


def add_rmsnorm(x, residual, weight, eps):
    """(s, n) in float64."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    n = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    if weight is not None:
        n = n * np.asarray(weight, np.float64)
    return s, n


def _order(values):
    """Indices by value, largest first, ties to the lower index."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))


def route_scored(logits, bias, top_k, score="softmax", groups=1, top_groups=1, group_rank=1, renormalize=False,
                 scale=1.0):
    """(ids, weights float64); masked experts (logit -inf or NaN) have no score."""
    T, E = logits.shape
    ids = np.zeros((T, top_k), np.int32)
    w = np.zeros((T, top_k), np.float64)
    for t in range(T):
        l = [float(v) for v in logits[t]]
        live = [not (math.isnan(v) or v == -math.inf) for v in l]
        sc = [0.0] * E
        if any(live):
            m = max(v for v, ok in zip(l, live) if ok)
            if score == "softmax":
                ex = [(1.0 if v == m else math.exp(v - m)) if ok else 0.0 for v, ok in zip(l, live)]
                tot = math.fsum(ex)
                sc = [v / tot for v in ex]
            else:
                sc = [(1 / (1 + math.exp(-v)) if v > -700 else math.exp(v) if v > -745 else 0.0) if ok else 0.0
                      for v, ok in zip(l, live)]
        choice = [s if ok else -math.inf for s, ok in zip(sc, live)]
        if bias is not None:
            choice = [c + float(b) if c != -math.inf and not math.isnan(b) else -math.inf
                      for c, b in zip(choice, bias)]
        if groups > 1:
            per = E // groups
            val = []
            for g in range(groups):
                best = sorted((c for c in choice[g * per:(g + 1) * per] if c != -math.inf), reverse=True)[:group_rank]
                val.append(sum(best) if best else -math.inf)
            kept = set(_order(val)[:top_groups])
            choice = [c if e // per in kept else -math.inf for e, c in enumerate(choice)]
        order = _order(choice)[:top_k]
        got = [sc[e] if choice[e] != -math.inf else 0.0 for e in order]
        tot = math.fsum(got)
        if renormalize:
            got = [g / tot if tot > 0 else 0.0 for g in got]
        ids[t] = order
        w[t] = [g * scale for g in got]
    return ids, w


def erf(a):
    return np.vectorize(math.erf, otypes=[np.float64])(a)


def silu(a):
    return a * 0.5 * (1 + np.tanh(0.5 * a))


def activate(a, act):
    if act == "relu":
        return np.maximum(a, 0)
    if act == "gelu":
        return 0.5 * a * (1 + erf(a / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * a * (1 + np.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    if act == "silu":
        return silu(a)
    return a


def linear(x, w, x_scale=None, w_scale=None, bias=None, act="none", residual=None):
    """(out, preactivation, sum of |products| scaled like it), all float64."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    a, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if x_scale is not None:
        f = np.outer(np.asarray(x_scale, np.float64), np.asarray(w_scale, np.float64))
        a, mag = a * f, mag * np.abs(f)
    if bias is not None:
        a = a + np.asarray(bias, np.float64)
    if act == "swiglu":
        n = w.shape[0] // 2
        out = silu(a[:, :n]) * a[:, n:]
    else:
        out = activate(a, act)
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
    return out, a, mag

"""The activations of moe_w4a16_linear by themselves: the product is 0 and the
bias is the argument, so FP32 outputs show the activation's own error.

u = 2^-24 is one FP32 rounding.  Bounds of the relative error, in u:
  SiLU       e^-a: |a| 2 (a log2 e and its constant) + 4 (2 ulp); the sum 1,
             the reciprocal 2, the product 1               -> 2 |a| + 8
  tanh GELU  its exponent E = 2 sqrt(2/pi) (|a| + 0.044715 |a|^3) takes 9
             roundings, the rest as SiLU                   -> 9 E + 8
  GELU       the tail's fit 4.2e-6 = 70, its exponent a^2/2 3 roundings, the
             exponential 4, t 3 times at most 3 (its effect on t p(t)), p
             1.75 (the sum of its terms' sizes over p) times 13, products 3
                                                           -> 110 + 1.5 a^2
SwiGLU as SiLU.  The ranges end where e^-E would leave FP32's range.
"""
import math

import numpy as np
import pytest
import torch

from w4a16_compact_expert_gb300 import block as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def reference(act, a):
    if act == "gelu":
        return 0.5 * a * np.vectorize(math.erfc)(-a / math.sqrt(2)), 110 + 1.5 * a * a
    if act == "gelu_tanh":
        e = 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        return a / (1 + np.exp(-e)), 9 * np.abs(e) + 8
    return a / (1 + np.exp(-a)), 2 * np.abs(a) + 8


@pytest.mark.parametrize("act,lo,hi", [("gelu", -12.0, 12.0), ("gelu_tanh", -9.5, 9.5), ("silu", -80.0, 80.0),
                                       ("swiglu", -80.0, 80.0)])
@pytest.mark.parametrize("T", [1, 40, 70])
def test_relative_error(act, lo, hi, T):
    g = torch.Generator().manual_seed(T)
    a = torch.cat([torch.linspace(lo, hi, 3001), torch.randn(1000, generator=g).clamp(lo, hi) * 2,
                   torch.tensor([1e-30, -1e-30, 1e-4, -1e-4])]).clamp(lo, hi)
    N = a.numel()
    x = torch.zeros(T, 8, dtype=torch.float16, device="cuda")
    w = torch.zeros(2 * N if act == "swiglu" else N, 8, dtype=torch.float16, device="cuda")
    bias = torch.cat([a, torch.ones(N)]) if act == "swiglu" else a
    out = B.linear(x, w, bias=bias.cuda(), act=act, out_dtype=torch.float32).double().cpu().numpy()
    ref, bound = reference(act, a.double().numpy())
    err = np.abs(out - ref)
    worst = (err / (np.abs(ref) * U)).max(0)
    assert (err <= bound * U * np.abs(ref)).all(), (act, float(worst.max()), float(a[int(worst.argmax())]))


def test_far_out():
    """Beyond those ranges the result is a, or 0 where its size is below 2^-119."""
    far = torch.tensor([1e3, 3e4, 1e30, -1e3, -3e4, -1e30, -100.0, 0.0, -0.0])
    x, w = torch.zeros(2, 8, dtype=torch.float16, device="cuda"), torch.zeros(9, 8, dtype=torch.float16, device="cuda")
    for act in ("gelu", "gelu_tanh", "silu"):
        out = B.linear(x, w, bias=far.cuda(), act=act, out_dtype=torch.float32).cpu()
        assert torch.equal(out[:, :3], far[:3].expand(2, 3)) and (out[:, 3:] == 0).all()

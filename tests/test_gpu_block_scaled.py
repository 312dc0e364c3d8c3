"""The block-scaled 8-bit path on the GPU against the float64 oracle.

Tolerances are error bounds, not fits.  u(t) = eps(t) / 2 is one rounding to
type t.  Norm: under 64 FP32 roundings, 2^-18 (as the norm with a scale per
row); a scale adds two.
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

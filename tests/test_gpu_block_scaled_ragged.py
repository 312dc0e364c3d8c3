"""linear_blocks where a warp's 32 tokens end inside the batch and its rows are stored from the lanes that hold them:
each token's outputs are the bits that a batch of whole warps gives it, and nothing is written behind the last."""
import pytest
import torch

from tests.test_gpu_block_scaled import BF16, E4, F16, F32, check_linear, make_linear, run
from w4a16_compact_expert_gb300 import block as B
from w4a16_compact_expert_gb300 import moe_w4a16 as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out,residual", [(F16, False), (F16, True), (BF16, False), (F32, True), (F32, False), (E4, False)])
@pytest.mark.parametrize("act,N", [("swiglu", 384), ("none", 512)])
def test_partial_warps(act, N, out, residual):
    x, w, xs, ws, b, r = make_linear(768, N, 400, act, True, residual, out, 3)
    parts = lambda o: o if isinstance(o, tuple) else (o,)   # noqa: E731
    bits = lambda t: t.contiguous().view(torch.uint8)   # noqa: E731
    whole = parts(run((x, w, xs, ws, b, r), act, out_dtype=out))
    for T in (65, 66, 95, 97, 127, 129, 255, 257, 287, 300, 511, 513, 545):
        buf = torch.full((T + 40, N), 3.0, device="cuda").to(out)   # rows on the 32-byte grid
        got = parts(B.linear_blocks(x[:T], w, xs[:T], ws, bias=b, act=act, residual=None if r is None else r[:T], out=buf[:T]))
        assert (buf[T:].float() == 3).all()
        assert all(torch.equal(bits(g), bits(o[:T])) for g, o in zip(got, whole)), T
    cut = None if r is None else r[:545]
    check_linear(x[:545], w, xs[:545], ws, b, cut, act, got if out is E4 else got[0])
    assert B.status() == F.OK

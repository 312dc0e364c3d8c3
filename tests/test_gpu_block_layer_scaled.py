"""A whole block whose shared expert is in E4M3 with a scale per 128 x 128 block, on the GPU."""
import numpy as np
import pytest

from oracle import block_oracle as BO
from tests import gpu_parity as gp
from tests.test_gpu_block_layer import oracle_routed
from w4a16_compact_expert_gb300 import moe_w4a16 as F, synth

pytestmark = pytest.mark.gpu


def squares(torch, a):
    """a [N, K] in E4M3 with a scale per 128 x 128 block."""
    N, K = a.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.nn.functional.pad(a, (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128)
    s = p.abs().amax((1, 3)) / 448
    q = (p / s[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)
    return q[:N, :K].contiguous(), s


@pytest.mark.parametrize("T", [1, 5, 33, 70, 300])
def test_block_with_a_block_scaled_shared_expert(T):
    """Against the oracle on the block's own routing and norm; the quantised intermediate is checked to its rounding."""
    import torch

    from w4a16_compact_expert_gb300 import block as B
    layer = synth.make_layer(synth.TINY, 31)
    H, I, k = layer.shape.hidden, 208, layer.shape.top_k
    m = gp.make_handle(layer, T)
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std   # noqa: E731
    x, res, nw, rw = rnd(T, H).half(), rnd(T, H).half(), (1 + rnd(H, std=0.1)).half(), rnd(layer.shape.num_experts, H, std=0.05).half()
    gate, gs = squares(torch, rnd(I, H, std=0.05))
    up, us = squares(torch, rnd(I, H, std=0.05))
    down, ds = squares(torch, rnd(H, I, std=0.05))
    gu, gus = torch.cat((gate.view(torch.uint8), up.view(torch.uint8))).view(torch.float8_e4m3fn), torch.cat((gs, us))
    try:
        blk = B.MoEBlock(m, nw, rw, shared=(gu, down), shared_scale=(gus, ds), renormalize=True)
        out, s = blk(x, res)
        n, s2, q, qs = B.add_rmsnorm(x, res, nw, quant="blocks")
        assert torch.equal(s, s2)
        ids, w = B.route_scored(B.linear(n, rw, out_dtype=torch.float32), k, renormalize=True)
        h, hs = B.linear_blocks(q, gu, qs, gus, act="swiglu", out_dtype=torch.float8_e4m3fn)
        f64 = lambda t: t.double().cpu().numpy()   # noqa: E731
        routed = oracle_routed(layer, n.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy())
        ref = routed + BO.linear_blocks(f64(h.float()), f64(down.float()), f64(hs), f64(ds))[0]
        got = f64(out)
        assert np.linalg.norm(got - ref) <= gp.TOL_NORM * np.linalg.norm(ref)
        assert np.abs(got - ref).max() <= gp.TOL_MAX * np.abs(ref).max()
        # the intermediate: half a step of E4M3 of every value, and the roundings before it
        v = BO.linear_blocks(f64(q.float()), f64(gu.float()), f64(qs), f64(gus), act="swiglu")[0]
        back = f64(h.float()) * np.repeat(f64(hs), 128, 1)[:, :I]
        step = np.repeat(f64(hs), 128, 1)[:, :I] * 2.0 ** -10
        assert (np.abs(back - v) <= 2.0 ** -4 * 1.001 * np.abs(v) + 1.001 * step + 1e-5 * np.abs(v).max()).all()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        other, _ = blk(x, res, stream=side)
        side.synchronize()
        assert torch.equal(other, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again, _ = blk(x, res)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)
        assert m.get_status() == (F.OK, 0) and B.status() == F.OK
    finally:
        m.close()


def test_block_refuses_mismatched_scales():
    import torch

    from w4a16_compact_expert_gb300 import block as B
    gu, dn = torch.zeros(256, 128, device="cuda").to(torch.float8_e4m3fn), torch.zeros(128, 128, device="cuda").half()
    for shared, scale in (((gu.half(), dn), (1, 2)), ((gu, dn), None), ((gu, dn), (1,)), ((gu, dn), [1, 2, 3]), (None, (1, 2))):
        with pytest.raises(ValueError):
            B.MoEBlock(None, None, None, shared=shared, shared_scale=scale)

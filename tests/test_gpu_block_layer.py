"""The layer's experts on given routing, and the whole block, on the GPU."""
import numpy as np
import pytest

from oracle import block_oracle as BO
from oracle import moe_oracle
from tests import gpu_parity as gp
from w4a16_compact_expert_gb300 import moe_w4a16 as F, synth

pytestmark = pytest.mark.gpu


def oracle_routed(layer, x, ids, w, residual=False):
    """sum_j w_j y(ids_j) in float64; absent experts and ids out of range contribute 0."""
    gq, gs, uq, us, dq, ds = layer.slot_experts().arrays()
    x = np.asarray(x, np.float64)
    T, k = ids.shape
    out = x.copy() if residual else np.zeros_like(x)
    for e in np.unique(ids):
        if not 0 <= e < layer.shape.num_experts or layer.expert_to_slot[e] < 0:
            continue
        s = int(layer.expert_to_slot[e])
        W = [moe_oracle.dequantize(a[s], b[s]) for a, b in ((gq, gs), (uq, us), (dq, ds))]
        t, j = np.nonzero(ids == e)
        y = moe_oracle.expert_ffn(x[t], *W)
        np.add.at(out, t, np.asarray(w, np.float64)[t, j][:, None] * y)
    return out


@pytest.fixture(scope="module")
def tiny():
    layer = synth.tiny_layer()
    m = gp.make_handle(layer, 700)
    yield layer, m
    m.close()


@pytest.mark.parametrize("T,force", [(1, 0), (3, 0), (12, F.FORCE_GEMV), (12, F.FORCE_GEMM), (70, 0), (70, F.FORCE_GEMV),
                                     (600, 0), (700, F.FORCE_GEMM)])
def test_routed_equals_the_router_path(tiny, T, force):
    """With the router's own ids and weights the bits are those of forward's separate launches."""
    import torch
    layer, m = tiny
    x = gp.to_dev(synth.draw_x(5, T, layer.shape.hidden))
    rw = gp.to_dev(layer.router_w)
    unfused = 0 if force == F.FORCE_GEMM or (force == 0 and T > 40) else F.UNFUSED
    ref, dbg = m.forward(x, rw, None, force | unfused, debug=True)
    out = m.forward_routed(x, dbg["ids"], dbg["weights"], force)
    path, launches = m.last_path()
    assert path == (F.PATH_DECODE if unfused or force == F.FORCE_GEMV else F.PATH_GEMM) and launches >= 3
    assert torch.equal(out, ref)
    assert m.get_status() == (F.OK, 0)


@pytest.mark.parametrize("T", [1, 5, 33, 130, 650])
@pytest.mark.parametrize("residual", [False, True])
def test_routed_against_the_oracle(tiny, T, residual):
    """Routing no router would give: repeated experts, one expert for all, negative and zero weights."""
    layer, m = tiny
    rng = np.random.default_rng(T)
    x = synth.draw_x(6, T, layer.shape.hidden)
    ids = rng.integers(0, 8, (T, 2)).astype(np.int32)
    ids[::3] = 5
    w = rng.standard_normal((T, 2)).astype(np.float32)
    w[::4, 1] = 0
    out = m.forward_routed(gp.to_dev(x), gp.to_dev(ids), gp.to_dev(w), F.RESIDUAL if residual else 0)
    ref = oracle_routed(layer, x, ids, w, residual)
    gp.assert_output(out.float().cpu().numpy().astype(np.float64), ref, np.ones(T, bool))
    assert m.get_status() == (F.OK, 0)


@pytest.mark.parametrize("T,force", [(4, 0), (90, F.FORCE_GEMM), (600, F.FORCE_GEMM)])
def test_routed_absent_experts_and_bad_ids(T, force):
    layer = synth.make_layer(synth.TINY, 77, num_resident=5)
    m = gp.make_handle(layer, T)
    try:
        rng = np.random.default_rng(1)
        x = synth.draw_x(8, T, 256)
        ids = rng.integers(0, 8, (T, 2)).astype(np.int32)
        w = np.full((T, 2), 0.5, np.float32)
        # every id in range: exactly the pairs of absent experts are missed
        out = m.forward_routed(gp.to_dev(x), gp.to_dev(ids), gp.to_dev(w), force)
        miss = int((layer.expert_to_slot[ids] < 0).sum())
        assert m.get_status() == ((F.ERR_NOT_RESIDENT if miss else F.OK), miss)
        gp.assert_output(out.float().cpu().numpy().astype(np.float64), oracle_routed(layer, x, ids, w), np.ones(T, bool))
        # ids out of range: weight 0, counted (as expert 0 once more if that is absent)
        bad = ids.copy()
        bad[0, 0], bad[T // 2, 1], bad[T - 1, 0] = -1, 8, 2 ** 31 - 1
        nbad = int(((bad < 0) | (bad > 7)).sum())
        out = m.forward_routed(gp.to_dev(x), gp.to_dev(bad), gp.to_dev(w), force)
        st, got = m.get_status()
        miss = sum(1 for e in bad.reshape(-1) if 0 <= e < 8 and layer.expert_to_slot[e] < 0)
        assert st == F.ERR_NOT_RESIDENT and miss + nbad <= got <= miss + 2 * nbad
        gp.assert_output(out.float().cpu().numpy().astype(np.float64), oracle_routed(layer, x, bad, w), np.ones(T, bool))
    finally:
        m.close()


@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9])
@pytest.mark.parametrize("force", [F.FORCE_GEMV, F.FORCE_GEMM])
def test_routed_one_expert_takes_every_pair(T, force):
    """Up to k pairs of a token for one expert: repeated ids, and ids out of range (taken as expert 0)."""
    layer = synth.make_layer(synth.LayerShape(hidden=2048, inter=256, num_experts=16, top_k=8), 78)
    m = gp.make_handle(layer, 9)
    try:
        x = synth.draw_x(9, T, 2048)
        w = np.full((T, 8), 0.125, np.float32)
        for ids in (np.full((T, 8), 3), np.where(np.arange(8) < 5, 0, -1) + np.zeros((T, 1), int), np.full((T, 8), 16)):
            ids = ids.astype(np.int32)
            bad = int(((ids < 0) | (ids > 15)).sum())
            out = m.forward_routed(gp.to_dev(x), gp.to_dev(ids), gp.to_dev(w), force)
            assert m.get_status() == ((F.ERR_NOT_RESIDENT, bad) if bad else (F.OK, 0))
            gp.assert_output(out.float().cpu().numpy().astype(np.float64), oracle_routed(layer, x, ids, w),
                             np.ones(T, bool))
    finally:
        m.close()


def test_routed_refusals(tiny):
    import torch
    _, m = tiny
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for flags in (F.PRENORM, F.OFFLOAD, F.UNFUSED, F.FORCE_GEMV | F.FORCE_GEMM):
        with pytest.raises(F.MoEError):
            m.forward_routed(x, ids, w, flags)
    with pytest.raises(F.MoEError):
        m.forward_routed(x, ids, w, out=x)
    for bad in ((x, ids.long(), w), (x, ids, w.double()), (x, ids[:3], w), (x[:, :128], ids, w), (x.float(), ids, w)):
        with pytest.raises(ValueError):
            m.forward_routed(*bad)
    assert m.forward_routed(x[:0], ids[:0], w[:0]).shape == (0, 256)


@pytest.mark.parametrize("T", [1, 9, 50, 300])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", True)])
def test_block(T, bits, score, bias):
    """The whole block against float64 of the GPU's own norm and routing (each has its own test)."""
    import torch
    from w4a16_compact_expert_gb300 import block as B
    shape = synth.LayerShape(hidden=256, inter=128, num_experts=16, top_k=4)
    layer = synth.make_layer(shape, 11)
    m = gp.make_handle(layer, 300)
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()   # noqa: E731
    x, res = rnd(T, 256).half(), rnd(T, 256).half()
    nw = (1 + rnd(256, std=0.1)).half()
    rw, gu, dn = rnd(16, 256, std=0.06).half(), rnd(384, 256, std=0.06), rnd(256, 192, std=0.07).half()
    b = rnd(16, std=0.1) if bias else None
    scale = gu.abs().amax(1) / 448 if bits == 8 else None
    gu = (gu / scale[:, None]).to(torch.float8_e4m3fn) if bits == 8 else gu.half()
    opts = dict(score=score, renormalize=True, groups=4, top_groups=2, group_rank=2, scale=1.5)
    try:
        blk = B.MoEBlock(m, nw, rw, shared=(gu, dn), shared_scale=scale, bias=b, **opts)
        out, s = blk(x, res)
        n, s2, q, qs = B.add_rmsnorm(x, res, nw, quant=bits == 8)
        assert torch.equal(s, s2)
        logits = B.linear(n, rw, out_dtype=torch.float32)
        ids, w = B.route_scored(logits, 4, bias=b, **opts)
        routed = oracle_routed(layer, n.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy())
        f64 = lambda t: None if t is None else t.double().cpu().numpy()   # noqa: E731
        h = BO.linear(f64((q if bits == 8 else n).float()), f64(gu.float()), f64(qs), f64(scale), act="swiglu")[0]
        ref = routed + h @ f64(dn).T
        got = f64(out)
        assert np.linalg.norm(got - ref) <= gp.TOL_NORM * np.linalg.norm(ref)
        assert np.abs(got - ref).max() <= gp.TOL_MAX * np.abs(ref).max()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again, _ = blk(x, res)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)
        assert m.get_status() == (F.OK, 0) and B.status() == F.OK
    finally:
        m.close()


@pytest.mark.parametrize("T,force", [(1, F.FORCE_GEMV), (4, F.FORCE_GEMV), (12, F.FORCE_GEMV), (4, F.FORCE_GEMM),
                                     (90, F.FORCE_GEMM)])
def test_routed_bad_ids_contribute_exactly_nothing(T, force):
    """Also where expert 0's output is not finite, or expert 0 is absent (each bad id is one miss)."""
    layer = synth.make_layer(synth.TINY, 79)
    rng = np.random.default_rng(T)
    x = synth.draw_x(9, T, 256)
    ids = rng.integers(1, 8, (T, 2)).astype(np.int32)
    ids[::2, 1] = np.array([-1, 8, 2 ** 31 - 1, -2 ** 31])[np.arange((T + 1) // 2) % 4]
    w = rng.standard_normal((T, 2)).astype(np.float32)
    bad = int(((ids < 0) | (ids > 7)).sum())
    ref = oracle_routed(layer, x, ids, w)
    m = F.MoELayer(256, 128, 8, 2, num_slots=8, max_tokens=T)
    try:
        gq, gs, uq, us, dq, ds = (a.copy() for a in layer.slot_experts().arrays())
        us[0] = 0x7E00   # NaN
        m.pack_experts(0, gq, gs, uq, us, dq, ds)
        for absent in (False, True):
            m.set_slot_table(np.array([-1 if absent else 0, 1, 2, 3, 4, 5, 6, 7], np.int32))
            out = m.forward_routed(gp.to_dev(x), gp.to_dev(ids), gp.to_dev(w), force)
            assert m.get_status() == (F.ERR_NOT_RESIDENT, bad)
            gp.assert_output(out.float().cpu().numpy().astype(np.float64), ref, np.ones(T, bool))
    finally:
        m.close()


@pytest.mark.parametrize("force", [F.FORCE_GEMV, F.FORCE_GEMM])
def test_routed_weight_zero_contributes_exactly_nothing(force):
    layer = synth.make_layer(synth.TINY, 80)
    x = synth.draw_x(9, 6, 256)
    ids = np.array([[0, 3]] * 6, np.int32)
    w = np.array([[0.0, 0.5], [-0.0, 1.0]] * 3, np.float32)
    m = F.MoELayer(256, 128, 8, 2, num_slots=8, max_tokens=6)
    try:
        gq, gs, uq, us, dq, ds = (a.copy() for a in layer.slot_experts().arrays())
        us[0] = 0x7E00   # NaN
        m.pack_experts(0, gq, gs, uq, us, dq, ds)
        m.set_slot_table(layer.expert_to_slot)
        out = m.forward_routed(gp.to_dev(x), gp.to_dev(ids), gp.to_dev(w), force)
        assert m.get_status() == (F.OK, 0)
        gp.assert_output(out.float().cpu().numpy().astype(np.float64), oracle_routed(layer, x, ids, w), np.ones(6, bool))
    finally:
        m.close()


def test_routed_output_is_allocated_for_the_stream(tiny, monkeypatch):
    import torch
    layer, m = tiny
    x, ids, w = gp.to_dev(synth.draw_x(5, 4, 256)), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.ones(4, 2).cuda()
    torch.cuda.synchronize()
    side, seen = torch.cuda.Stream(), []
    empty_like = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t: (seen.append(torch.cuda.current_stream()), empty_like(t))[1])
    out = m.forward_routed(x, ids, w, stream=side)
    side.synchronize()
    assert seen == [side]
    assert torch.equal(out, m.forward_routed(x, ids, w))
    torch.cuda.synchronize()
    assert seen == [side, torch.cuda.current_stream()]

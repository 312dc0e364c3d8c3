"""One decoder block's feed-forward half on the GPU, with synthetic weights:
residual addition and norm, router with renormalised top-8 weights, 64 routed
INT4 experts, and a shared expert whose gate and up run in E4M3.

  python examples/moe_block.py [tokens ...]

prints the time of a block per token count, captured in a CUDA graph as a
decode loop would run it (weights of one block; they stay in L2 where they
fit), and how far the output is from the same block in FP32 on a few tokens.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from w4a16_compact_expert_gb300 import block, synth  # noqa: E402
from w4a16_compact_expert_gb300.moe_w4a16 import MoELayer  # noqa: E402


def make_block(shape=synth.OLMOE, shared_inter=1024, seed=7, max_tokens=2048):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, E = shape.hidden, shape.num_experts

    def normal(*s, std=0.02):
        return torch.randn(*s, device="cuda", generator=g) * std

    layer = MoELayer(H, shape.inter, E, shape.top_k, max_tokens=max_tokens)
    experts = synth.device_random_experts(shape, E, seed, "cuda")
    layer.pack_experts(0, *experts)
    layer.set_slot_table(range(E))
    gate_up = normal(2 * shared_inter, H)
    scale = gate_up.abs().amax(1) / 448
    return block.MoEBlock(
        layer, (1 + normal(H, std=0.1)).half(), normal(E, H).half(),
        shared=((gate_up / scale[:, None]).to(torch.float8_e4m3fn), normal(H, shared_inter).half()),
        shared_scale=scale, score="softmax", renormalize=True), experts


def reference(b, experts, x, residual):
    """The block in FP32, token by token, from the packed experts."""
    s = x.float() + residual.float()
    n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + b.eps) * b.norm_weight.float()
    p = torch.softmax(n @ b.router_w.float().t(), -1)
    w, ids = p.topk(b.layer.cfg.top_k, -1)
    w = w / w.sum(-1, keepdim=True)

    def dense(q, sc):
        lo, hi = (q & 15).short(), (q >> 4).short()
        v = torch.stack((lo, hi), -1).flatten(-2).float()
        v = torch.where(v > 7, v - 16, v)
        return v * sc.view(torch.float16).float().repeat_interleave(256, -1)[..., :v.shape[-1]]

    out = torch.zeros_like(s)
    for t in range(x.shape[0]):
        for e, we in zip(ids[t].tolist(), w[t].tolist()):
            gq, gs, uq, us, dq, ds = (a[e] for a in experts)
            h = torch.nn.functional.silu(dense(gq, gs) @ n[t]) * (dense(uq, us) @ n[t])
            out[t] += we * (dense(dq, ds) @ h)
    gu = n @ (b.gate_up.float() * b.scale[:, None]).t()
    gate, up = gu.chunk(2, -1)
    return out + (torch.nn.functional.silu(gate) * up) @ b.down.float().t()


def main(tokens):
    b, experts = make_block(max_tokens=max(tokens))
    for T in tokens:
        x, r = torch.randn(T, 2048, device="cuda").half(), torch.randn(T, 2048, device="cuda").half()
        out, _ = b(x, r)
        ref = reference(b, experts, x[:4], r[:4])
        err = ((out[:4].float() - ref).norm() / ref.norm()).item()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                b(x, r)
        g.replay()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(10):
            g.replay()
        t1.record()
        torch.cuda.synchronize()
        print(f"T={T:5d}  {t0.elapsed_time(t1) * 5:8.1f} us per block, "
              f"{T / (t0.elapsed_time(t1) * 5e-6):12.0f} tokens/s, off FP32 by {err:.1e} (8-bit gate and up included)")
    assert b.layer.get_status()[0] == 0 and block.status() == 0


if __name__ == "__main__":
    main([int(a) for a in sys.argv[1:]] or [1, 4, 16, 64, 256, 2048])

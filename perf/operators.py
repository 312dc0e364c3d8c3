"""Cases of the operators that stand around the routed experts of one block.

  norm    s = x + residual; y = s / rms(s) * weight; q = y in e4m3 with one scale per row
  route   scores of router logits (softmax or sigmoid), selection bias, groups, top-k, renormalised weights
  linear  act(x W^T * scales + bias) + residual: the router product and the shared expert's two products

`run` computes a pass in plain torch operations, or, where `own` is true, by
the framework's calls.  Inputs have the distributions of the synthetic layers:
activations N(0, 1), weights N(0, 0.02).
"""
import functools
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one decoded token between two layers, normalised for the experts and quantised for the shared expert
        {"name": "norm_token", "op": "norm", "T": 1, "H": 2048, "dtype": "fp16", "residual": True, "quant": True},
        # a prompt of 2048 tokens through the same place
        {"name": "norm_prompt", "op": "norm", "T": 2048, "H": 2048, "dtype": "fp16", "residual": True, "quant": True},
        # a long batch of a wider model in bf16, the first layer (nothing to add), an odd row count
        {"name": "norm_long", "op": "norm", "T": 16383, "H": 4096, "dtype": "bf16", "residual": False, "quant": False},
        # one decoded token over 64 experts, weights renormalised
        {"name": "route_token", "op": "route", "T": 1, "E": 64, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "rank": 1, "renorm": True, "scale": 1.0, "dtype": "fp32"},
        # a prompt over 60 experts, top-4, weights as they come out of the softmax
        {"name": "route_prompt", "op": "route", "T": 2048, "E": 60, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "rank": 1, "renorm": False, "scale": 1.0, "dtype": "fp32"},
        # a long batch over 256 experts in 8 groups with a balancing bias
        {"name": "route_groups", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "rank": 2, "renorm": True, "scale": 2.5, "dtype": "fp32"},
        # the router's logits of a decode batch
        {"name": "linear_router", "op": "linear", "T": 16, "N": 64, "K": 2048, "dtype": "fp16", "out": "fp32",
         "act": "none", "bias": False, "residual": False},
        # one token through the shared expert: gate and up, then down onto the residual stream
        {"name": "linear_token_gated", "op": "linear", "T": 1, "N": 5632, "K": 2048, "dtype": "fp16", "out": "fp16",
         "act": "swiglu", "bias": False, "residual": False},
        {"name": "linear_batch_down", "op": "linear", "T": 32, "N": 2048, "K": 5632, "dtype": "fp16", "out": "fp16",
         "act": "none", "bias": False, "residual": True},
        # a ragged middle batch of a dense layer with bias and gelu
        {"name": "linear_ragged", "op": "linear", "T": 333, "N": 4001, "K": 1416, "dtype": "bf16", "out": "bf16",
         "act": "gelu", "bias": True, "residual": False},
        # a prompt through the shared expert: 8-bit gate and up, 16-bit down
        {"name": "linear_prompt_8bit", "op": "linear", "T": 2048, "N": 5632, "K": 2048, "dtype": "e4m3",
         "out": "fp16", "act": "swiglu", "bias": False, "residual": False},
        {"name": "linear_prompt_down", "op": "linear", "T": 4096, "N": 2048, "K": 5632, "dtype": "fp16",
         "out": "fp16", "act": "none", "bias": True, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "linear", "linear"])
    if op == "norm":
        T = _log_int(rng, 1, 16384)
        H = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)])
        H = max(1, min(H, (16383 * 4096) // T))
        return {"op": op, "T": T, "H": H, "dtype": rng.choice(["fp16", "bf16"]), "residual": rng.random() < 0.7,
                "quant": rng.random() < 0.5}
    if op == "route":
        G, per = rng.choice([(1, rng.randint(8, 256)), (rng.choice([2, 4, 8]), rng.choice([8, 16, 20, 32]))])
        E = G * per
        tg = rng.randint(1, G)
        k = rng.randint(1, min(10, tg * per))
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": G, "top_groups": tg, "rank": rng.choice([1, 2]),
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "dtype": rng.choice(["fp32", "fp32", "fp16", "bf16"])}
    dtype = rng.choice(["fp16", "fp16", "bf16", "e4m3"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
    T = _log_int(rng, 1, 4096)
    N = _log_int(rng, 33, 6000)
    K = 16 * _log_int(rng, 4, 352)
    most = 2 * 4096 * 2048 * 5632
    while (4 if act == "swiglu" else 2) * T * N * K > most:
        T = (T + 1) // 2
    out = "bf16" if dtype == "bf16" else rng.choice(["fp16", "bf16"]) if dtype == "e4m3" else "fp16"
    return {"op": op, "T": T, "N": N, "K": K, "dtype": dtype, "out": out, "act": act, "bias": rng.random() < 0.5,
            "residual": rng.random() < 0.5}


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        b = 2 * T * H * (2 + 2 * case["residual"]) + 2 * H + (T * H + 4 * T) * case["quant"]
        return {"bytes": b, "flops": 4 * T * H}
    if case["op"] == "route":
        b = T * case["E"] * torch.finfo(TYPES[case["dtype"]]).bits // 8 + 4 * case["E"] * case["bias"]
        return {"bytes": b + 8 * T * case["k"], "flops": 4 * T * case["E"]}
    N, K = case["N"], case["K"]
    M = 2 * N if case["act"] == "swiglu" else N
    size = 1 if case["dtype"] == "e4m3" else 2
    osize = 4 if case["out"] == "fp32" else 2
    b = size * (T * K + M * K) + osize * T * N * (1 + case["residual"]) + 4 * M * case["bias"]
    if case["dtype"] == "e4m3":
        b += 4 * (T + M)
    return {"bytes": b, "flops": 2 * T * M * K}


def _rows_e4m3(a):
    """Rows of a in e4m3 with one scale each, as a checkpoint or the norm holds them."""
    s = a.abs().amax(-1) / E4M3_MAX
    return (a / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=g) * std

    T, t = case["T"], TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        H = case["H"]
        s["x"] = normal(T, H).to(t)
        s["res"] = normal(T, H, std=2.0).to(t) if case["residual"] else None
        s["w"] = (1 + normal(H, std=0.1)).to(t)
        s["out"] = (torch.empty(T, H, device=dev, dtype=t),
                    torch.empty(T, H, device=dev, dtype=t) if case["residual"] else None,
                    torch.empty(T, H, device=dev, dtype=torch.float8_e4m3fn) if case["quant"] else None,
                    torch.empty(T, device=dev) if case["quant"] else None)
    elif case["op"] == "route":
        s["logits"] = normal(T, case["E"], std=0.9).to(t)   # x N(0, 1), W_r N(0, 0.02), 2048 products
        s["b"] = normal(case["E"], std=0.05) if case["bias"] else None
        s["out"] = (torch.empty(T, case["k"], device=dev, dtype=torch.int32),
                    torch.empty(T, case["k"], device=dev))
    else:
        N, K = case["N"], case["K"]
        M = 2 * N if case["act"] == "swiglu" else N
        x, w = normal(T, K), normal(M, K, std=0.02)
        s["xs"] = s["ws"] = None
        if case["dtype"] == "e4m3":
            s["x"], s["xs"] = _rows_e4m3(x)
            s["w"], s["ws"] = _rows_e4m3(w)
        else:
            s["x"], s["w"] = x.to(t), w.to(t)
        s["b"] = normal(M, std=0.1) if case["bias"] else None
        s["res"] = normal(T, N).to(TYPES[case["out"]]) if case["residual"] else None
        s["out_t"] = torch.empty(T, N, device=dev, dtype=TYPES[case["out"]])
    return s


def _norm(x, res, w, real):
    s = x.to(real) if res is None else x.to(real) + res.to(real)
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * w.to(real)
    return s, y


def _act(a, name):
    if name == "relu":
        return a.clamp_min(0)
    if name == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    if name == "silu":
        return a / (1 + torch.exp(-a))
    if name == "swiglu":
        gate, up = a.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    return a


def _first(values, n):
    """Places of the n largest of each row, largest first, ties to the lower place."""
    return torch.sort(values, dim=-1, descending=True, stable=True)[1][:, :n]


def _route(s):
    """In 64 bits: two choices may be nearer to each other than 32 bits tell apart."""
    E, G, k = s["E"], s["groups"], s["k"]
    logits = s["logits"].double()
    if s["score"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = p / p.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    choice = score if s["b"] is None else score + s["b"].double()
    if G > 1:
        each = choice.view(-1, G, E // G)
        group = torch.sort(each, dim=-1, descending=True)[0][..., :s["rank"]].sum(-1)
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, _first(group, s["top_groups"]), True)
        choice = torch.where(kept[..., None], each, -math.inf).view(-1, E)
    ids = _first(choice, k)
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.int(), (w * s["scale"]).float()


@functools.lru_cache(maxsize=None)
def _framework():
    from w4a16_compact_expert_gb300 import block
    return block


def run(state):
    s = state
    if own:
        block = _framework()
        if s["op"] == "norm":
            y, r, q, qs = block.add_rmsnorm(s["x"], s["res"], s["w"], eps=EPS, quant=s["quant"], out=s["out"])
            return {"y": y, "residual": r, "q": q, "q_scale": qs}
        if s["op"] == "route":
            ids, w = block.route_scored(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"],
                                        top_groups=s["top_groups"], group_rank=s["rank"], renormalize=s["renorm"],
                                        scale=s["scale"], out=s["out"])
            return {"ids": ids, "weights": w}
        return {"out": block.linear(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["res"],
                                    x_scale=s["xs"], w_scale=s["ws"], out=s["out_t"])}
    if s["op"] == "norm":
        r, y = _norm(s["x"], s["res"], s["w"], torch.float32)
        q = qs = None
        if s["quant"]:
            qs = y.abs().amax(-1) / E4M3_MAX
            q = (y / qs[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        t = s["x"].dtype
        return {"y": y.to(t), "residual": r.to(t) if s["residual"] else None, "q": q, "q_scale": qs}
    if s["op"] == "route":
        ids, w = _route(s)
        return {"ids": ids, "weights": w}
    a = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        a = a * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        a = a + s["b"]
    a = _act(a, s["act"])
    if s["res"] is not None:
        a = a + s["res"].float()
    return {"out": a.to(s["out_t"].dtype)}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        v = s["x"].double()
        if s["residual"]:
            v = s["res"].double() + v
        rms = (v.pow(2).sum(1) / s["H"] + EPS).sqrt()
        y = v / rms[:, None] * s["w"].double()
        # q has no such value: next to a border of e4m3 the last bit of y decides
        return {"y": y, "residual": v if s["residual"] else None, "q": None,
                "q_scale": y.abs().max(1).values / E4M3_MAX if s["quant"] else None}
    if s["op"] == "route":
        # the weights of the chosen experts, by sets instead of sorting: an expert is
        # chosen when fewer than k of its rivals come before it
        l = s["logits"].double()
        score = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
        c = score.clone()
        if s["bias"]:
            c += s["b"].double()
        T, E, G = s["T"], s["E"], s["groups"]
        n = torch.arange(E, device=l.device)
        out_i = torch.empty(T, s["k"], dtype=torch.int32, device=l.device)
        out_w = torch.empty(T, s["k"], dtype=torch.float64, device=l.device)

        def place(v):
            """How many come before each one of a row: larger, or equal and earlier."""
            i = torch.arange(v.shape[1], device=v.device)
            a, b = v[:, :, None], v[:, None, :]
            return ((b > a) | ((b == a) & (i[None, None, :] < i[None, :, None]))).sum(2)

        for t0 in range(0, T, 2048):
            ct, st = c[t0:t0 + 2048], score[t0:t0 + 2048]
            if G > 1:
                byg = ct.unflatten(1, (G, E // G))
                best = byg.topk(s["rank"], 2).values.sum(2)
                alive = place(best) < s["top_groups"]
                ct = ct.masked_fill(~alive.repeat_interleave(E // G, 1), -math.inf)
            pl = place(ct)
            for j in range(s["k"]):
                at = ((pl == j) * n).sum(1)
                out_i[t0:t0 + 2048, j] = at.int()
                out_w[t0:t0 + 2048, j] = st.gather(1, at[:, None])[:, 0]
        if s["renorm"]:
            out_w /= out_w.sum(1, keepdim=True)
        return {"ids": out_i, "weights": out_w * s["scale"]}
    acc = torch.einsum("tk,nk->tn", s["x"].double(), s["w"].double())
    if s["dtype"] == "e4m3":
        acc = acc * torch.outer(s["xs"].double(), s["ws"].double())
    if s["bias"]:
        acc += s["b"].double()[None]
    N = s["N"]
    name = s["act"]
    if name == "relu":
        acc = torch.where(acc > 0, acc, torch.zeros_like(acc))
    elif name == "gelu":
        acc = acc * (1 - 0.5 * torch.erfc(acc / math.sqrt(2)))
    elif name == "gelu_tanh":
        acc = acc * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (acc + 0.044715 * acc ** 3))
    elif name == "silu":
        acc = acc * torch.sigmoid(acc)
    elif name == "swiglu":
        acc = acc[:, :N] * torch.sigmoid(acc[:, :N]) * acc[:, N:]
    if s["residual"]:
        acc += s["res"].double()
    return {"out": acc}

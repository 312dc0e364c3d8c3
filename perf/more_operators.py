"""Cases of the block-scaled 8-bit path and of scoring tokens.

  norm      s = x + residual; n = s / rms(s) * weight; n in e4m3 with one scale per row and 128 values
  linear    act(x W^T + bias) + residual of e4m3 operands, x with a scale per row and 128 of K, W with one per
            128 x 128 block; the output in 16 or 32 bits, or in e4m3 with a scale per row and 128 values
  logprobs  log probability of each row's given token, the row's entropy, its k most likely tokens

`run` computes a pass in plain torch operations, or, where `own` is true, by
the framework's calls.  Activations are N(0, 1), weights N(0, 0.02), logits
as a head over normalised activations gives them, rounded to their type.
"""
import functools
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
EPS = 1e-6
BLOCK = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}


def listed():
    return [
        # one decoded token between two layers, normalised for the experts and quantised for the shared expert
        {"name": "norm_token", "op": "norm", "T": 1, "H": 2048, "dtype": "fp16", "residual": True},
        # a long batch of a wider model
        {"name": "norm_long", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "residual": True},
        # one token through the shared expert: gate and up, quantised for down
        {"name": "linear_token_gated", "op": "linear", "T": 1, "N": 5632, "K": 2048, "act": "swiglu", "out": "e4m3",
         "bias": False, "residual": False},
        # a decode batch through the output head
        {"name": "linear_batch_head", "op": "linear", "T": 8, "N": 50304, "K": 2048, "act": "none", "out": "fp32",
         "bias": False, "residual": False},
        # a larger decode batch through the shared expert's down, onto the residual stream
        {"name": "linear_batch_down", "op": "linear", "T": 32, "N": 2048, "K": 5632, "act": "none", "out": "fp16",
         "bias": False, "residual": True},
        # a ragged middle batch of a dense layer with bias and gelu, blocks that end inside
        {"name": "linear_ragged", "op": "linear", "T": 333, "N": 4001, "K": 1424, "act": "gelu", "out": "bf16",
         "bias": True, "residual": False},
        # a prompt through the shared expert: gate and up, then down
        {"name": "linear_prompt_gated", "op": "linear", "T": 2048, "N": 5632, "K": 2048, "act": "swiglu",
         "out": "e4m3", "bias": False, "residual": False},
        {"name": "linear_prompt_down", "op": "linear", "T": 4096, "N": 2048, "K": 5632, "act": "none", "out": "fp16",
         "bias": False, "residual": True},
        # one decoded token's log probability with its 20 best alternatives
        {"name": "logprobs_token", "op": "logprobs", "T": 1, "V": 50304, "dtype": "fp32", "k": 20, "masked": 0.0},
        # a decode batch over a larger vocabulary
        {"name": "logprobs_batch", "op": "logprobs", "T": 64, "V": 151936, "dtype": "fp32", "k": 5, "masked": 0.0},
        # a ragged batch over an odd vocabulary, part of it masked for each row
        {"name": "logprobs_ragged", "op": "logprobs", "T": 333, "V": 32003, "dtype": "bf16", "k": 8, "masked": 0.3},
        # the tokens of a long prompt, scored
        {"name": "logprobs_prompt", "op": "logprobs", "T": 4096, "V": 131072, "dtype": "bf16", "k": 0, "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "logprobs", "logprobs"])
    if op == "norm":
        T = _log_int(rng, 1, 16384)
        H = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)])
        return {"op": op, "T": T, "H": max(1, min(H, (8192 * 4096) // T)), "dtype": rng.choice(["fp16", "bf16"]),
                "residual": rng.random() < 0.7}
    if op == "logprobs":
        dtype = rng.choice(["fp32", "fp16", "bf16"])
        k = rng.choice([0, 1, 5, 20, rng.randint(2, 32)])
        V = _log_int(rng, 500, 200000)
        T = min(_log_int(rng, 1, 8192), ((1 << 27) if k else (1 << 28)) // V)
        return {"op": op, "T": T, "V": V, "dtype": dtype, "k": k, "masked": rng.choice([0.0, 0.0, 0.5, 0.95])}
    act = rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "swiglu"])
    T = _log_int(rng, 1, 4096)
    N = _log_int(rng, 33, 6000)
    K = 16 * _log_int(rng, 4, 352)
    while (4 if act == "swiglu" else 2) * T * N * K > 2 * 4096 * 2048 * 5632:
        T = (T + 1) // 2
    out = rng.choice(["fp16", "bf16", "fp32", "e4m3"])
    return {"op": op, "T": T, "N": N, "K": K, "act": act, "out": out, "bias": rng.random() < 0.5,
            "residual": out != "e4m3" and rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        return {"bytes": 2 * T * H * (2 + 2 * case["residual"]) + 2 * H + T * H + 4 * T * _blocks(H), "flops": 5 * T * H}
    if case["op"] == "logprobs":
        size = torch.finfo(TYPES[case["dtype"]]).bits // 8
        return {"bytes": T * case["V"] * size + 16 * T + 8 * T * case["k"], "flops": 5 * T * case["V"]}
    N, K = case["N"], case["K"]
    parts = 2 if case["act"] == "swiglu" else 1
    M = parts * N
    osize = torch.finfo(TYPES[case["out"]]).bits // 8
    b = T * K + M * K + 4 * _blocks(K) * (T + parts * _blocks(N)) + osize * T * N * (1 + case["residual"])
    return {"bytes": b + 4 * M * case["bias"] + (4 * T * _blocks(N) if case["out"] == "e4m3" else 0),
            "flops": 2 * T * M * K}


def _scaled(a, s):
    """a / s in e4m3; zeros where s is 0."""
    q = torch.where(s > 0, a / s, torch.zeros_like(a))
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)


def _rows_e4m3(a):
    """Rows of a [T, n] in e4m3 with a scale per 128 values: (q [T, n], scale [T, ceil(n / 128)])."""
    T, n = a.shape
    b = torch.nn.functional.pad(a, (0, _blocks(n) * BLOCK - n)).view(T, _blocks(n), BLOCK)
    s = b.abs().amax(-1) / E4M3_MAX
    return _scaled(b, s[..., None]).reshape(T, -1)[:, :n].contiguous(), s


def _squares_e4m3(a):
    """a [N, K] in e4m3 with a scale per 128 x 128 block, as a checkpoint holds it."""
    N, K = a.shape
    b = torch.nn.functional.pad(a, (0, _blocks(K) * BLOCK - K, 0, _blocks(N) * BLOCK - N))
    b = b.view(_blocks(N), BLOCK, _blocks(K), BLOCK)
    s = b.abs().amax((1, 3)) / E4M3_MAX
    q = _scaled(b, s[:, None, :, None]).reshape(_blocks(N) * BLOCK, -1)
    return q[:N, :K].contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=g) * std

    T = case["T"]
    s = dict(case)
    if case["op"] == "norm":
        H, t = case["H"], TYPES[case["dtype"]]
        s["x"] = normal(T, H).to(t)
        s["res"] = normal(T, H, std=2.0).to(t) if case["residual"] else None
        s["w"] = (1 + normal(H, std=0.1)).to(t)
        s["out"] = (torch.empty(T, H, device=dev, dtype=t),
                    torch.empty(T, H, device=dev, dtype=t) if case["residual"] else None,
                    torch.empty(T, H, device=dev, dtype=E4M3), torch.empty(T, _blocks(H), device=dev))
    elif case["op"] == "logprobs":
        V, k = case["V"], case["k"]
        x = normal(T, V, std=2.5)
        s["tokens"] = torch.randint(0, V, (T,), device=dev, generator=g)
        likely = torch.rand(T, device=dev, generator=g) < 0.5   # the other half of the tokens is nobody's guess
        s["tokens"] = torch.where(likely, x.argmax(-1), s["tokens"])
        if case["masked"]:
            off = torch.rand(T, V, device=dev, generator=g) < case["masked"]
            off.scatter_(1, s["tokens"][:, None], False)
            x.masked_fill_(off, -math.inf)
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["out"] = (torch.empty(T, device=dev), torch.empty(T, device=dev),
                    torch.empty(T, k, device=dev, dtype=torch.int32) if k else None,
                    torch.empty(T, k, device=dev) if k else None)
    else:
        N, K = case["N"], case["K"]
        s["x"], s["xs"] = _rows_e4m3(normal(T, K))
        if case["act"] == "swiglu":   # gate and up are two matrices with blocks of their own
            (qa, sa), (qb, sb) = _squares_e4m3(normal(N, K, std=0.02)), _squares_e4m3(normal(N, K, std=0.02))
            s["w"] = torch.cat((qa.view(torch.uint8), qb.view(torch.uint8))).view(E4M3)
            s["ws"] = torch.cat((sa, sb))
        else:
            s["w"], s["ws"] = _squares_e4m3(normal(N, K, std=0.02))
        s["b"] = normal(s["w"].shape[0], std=0.1) if case["bias"] else None
        t = TYPES[case["out"]]
        s["res"] = normal(T, N).to(t) if case["residual"] else None
        s["out_t"] = torch.empty(T, N, device=dev, dtype=t)
        s["out_s"] = torch.empty(T, _blocks(N), device=dev) if case["out"] == "e4m3" else None
    return s


def _spread(scale, n, dim=-1):
    """Each scale at its 128 places."""
    return scale.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _weights(s, real):
    """W in real numbers."""
    N, K, w = s["N"], s["K"], s["w"].to(real)
    f = _spread(s["ws"].to(real), K)
    if s["act"] == "swiglu":
        gate, up = f.chunk(2, 0)
        return w * torch.cat((_spread(gate, N, 0), _spread(up, N, 0)))
    return w * _spread(f, N, 0)


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


@functools.lru_cache(maxsize=None)
def _framework():
    from w4a16_compact_expert_gb300 import block
    return block


def _own(s):
    block = _framework()
    if s["op"] == "norm":
        y, r, q, qs = block.add_rmsnorm(s["x"], s["res"], s["w"], eps=EPS, quant="blocks", out=s["out"])
        return {"y": y, "residual": r, "q": q, "q_scale": qs}
    if s["op"] == "logprobs":
        logprob, entropy, ids, top = block.token_logprobs(s["logits"], s["tokens"], s["k"], out=s["out"])
        return {"logprob": logprob, "entropy": entropy, "ids": ids, "top": top}
    out = block.linear_blocks(s["x"], s["w"], s["xs"], s["ws"], bias=s["b"], act=s["act"], residual=s["res"],
                              out=s["out_t"], out_scale=s["out_s"])
    out, scale = out if s["out"] == "e4m3" else (out, None)
    return {"out": out, "scale": scale}


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "norm":
        t = s["x"].dtype
        r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
        y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["w"].float()
        q, qs = _rows_e4m3(y)
        return {"y": y.to(t), "residual": r.to(t) if s["residual"] else None, "q": q, "q_scale": qs}
    if s["op"] == "logprobs":
        x = s["logits"].float()
        d = x - x.amax(-1, keepdim=True)
        e = torch.exp(d)
        total = e.sum(-1)
        log_total = torch.log(total)
        entropy = log_total - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1) / total
        logprob = d.gather(1, s["tokens"][:, None])[:, 0] - log_total
        if not s["k"]:
            return {"logprob": logprob, "entropy": entropy, "ids": None, "top": None}
        ids = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :s["k"]]
        return {"logprob": logprob, "entropy": entropy, "ids": ids.int(), "top": d.gather(1, ids) - log_total[:, None]}
    a = (s["x"].float() * _spread(s["xs"], s["K"])) @ _weights(s, torch.float32).t()
    if s["b"] is not None:
        a = a + s["b"]
    a = _act(a, s["act"])
    if s["res"] is not None:
        a = a + s["res"].float()
    if s["out"] == "e4m3":
        q, scale = _rows_e4m3(a)
        return {"out": q, "scale": scale}
    return {"out": a.to(s["out_t"].dtype), "scale": None}


def _largest_of_blocks(v):
    """max |v| of every 128 values of a row, the last block as long as it is."""
    n = v.shape[1]
    whole = n // BLOCK * BLOCK
    parts = [v[:, :whole].unflatten(1, (-1, BLOCK)).abs().max(2).values] if whole else []
    return torch.cat(parts + ([v[:, whole:].abs().max(1, keepdim=True).values] if whole < n else []), 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        v = s["x"].double()
        if s["residual"]:
            v = s["res"].double() + v
        rms = (v.pow(2).sum(1) / s["H"] + EPS).sqrt()
        y = v / rms[:, None] * s["w"].double()
        # q has no such value: next to a border of e4m3 the last bit of y decides
        return {"y": y, "residual": v if s["residual"] else None, "q": None, "q_scale": _largest_of_blocks(y) / E4M3_MAX}
    if s["op"] == "logprobs":
        T, V, k = s["T"], s["V"], s["k"]
        lp = torch.empty(T, dtype=torch.float64, device="cuda")
        ent, ids = lp.clone(), torch.empty(T, k, dtype=torch.int32, device="cuda")
        top = torch.empty(T, k, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // V)
        back = torch.arange(V - 1, -1, -1, device="cuda")
        for t in range(0, T, step):
            raw = s["logits"][t:t + step]
            l = torch.log_softmax(raw.double(), 1)
            lp[t:t + step] = l.gather(1, s["tokens"][t:t + step, None])[:, 0]
            ent[t:t + step] = -torch.special.xlogy(l.exp(), l.exp()).sum(1)
            if k:
                # values and places in one whole number: larger first, then the earlier
                bits = raw.float().view(torch.int32).long()
                order = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 20) + back
                at = order.topk(k, 1).indices
                ids[t:t + step], top[t:t + step] = at.int(), l.gather(1, at)
        return {"logprob": lp, "entropy": ent, "ids": ids if k else None, "top": top if k else None}
    T, N, K = s["T"], s["N"], s["K"]
    w = s["w"].double()
    rows = N if s["act"] != "swiglu" else 2 * N
    acc = torch.zeros(T, rows, dtype=torch.float64, device="cuda")
    at = torch.arange(rows, device="cuda") % N // BLOCK
    if s["act"] == "swiglu":
        at[N:] += _blocks(N)
    for b in range(_blocks(K)):
        cut = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        part = s["x"][:, cut].double() @ w[:, cut].T
        acc.addcmul_(part * s["xs"][:, b, None].double(), s["ws"][at, b].double()[None].expand_as(part))
    if s["bias"]:
        acc += s["b"].double()[None]
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
    if s["out"] == "e4m3":
        return {"out": None, "scale": _largest_of_blocks(acc) / E4M3_MAX}
    return {"out": acc, "scale": None}

"""What a decode step needs between its blocks: cases, plain forms and 64-bit values.

Operators, and what a pass of each computes:

  norm     the norm after a block, its gate and scale, the sum with the residual, and the norm before the next block
  product  y = res + scale * act(x . W^T + bias) for bf16 weights W; bf16 or fp32 outputs
  sample   a token of every row of logits: temperature, top-k, top-p, min-p, and a given uniform number

``run`` computes the plain forms in float32 (the sampler's weights and their sums in float64), or calls the library
where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the sum with the residual and the norm before a block, one decoded token, H = 2048: latency
        {"name": "norm one token", "op": "norm", "n": 1, "heads": 0, "dim": 2048, "res": "bf16", "post": "", "pre": "rms",
         "gate": "", "scale": 1.0},
        # the norm of every query head of a decode batch: many short rows, no residual
        {"name": "norm heads", "op": "norm", "n": 32, "heads": 32, "dim": 128, "res": "", "post": "", "pre": "rms",
         "gate": "", "scale": 1.0},
        # the same sum and norm over prompts, H = 4096
        {"name": "norm prompts", "op": "norm", "n": 8192, "heads": 0, "dim": 4096, "res": "bf16", "post": "",
         "pre": "rms", "gate": "", "scale": 1.0},
        # norms on both sides of a block, H = 7168, its output gated per token and scaled, the residual kept in fp32
        {"name": "norm both sides gated", "op": "norm", "n": 3001, "heads": 0, "dim": 7168, "res": "f32",
         "post": "rms1", "pre": "rms1", "gate": "token", "scale": 0.22},
        # the fused q, k, v projection of one decoded token with its bias, H = 2048: latency
        {"name": "product one token", "op": "product", "n": 1, "N": 5120, "K": 2048, "bias": True, "act": "none",
         "res": False, "out": "bf16", "scale": 1.0},
        # gate and up rows of a shared expert for a decode batch, H = 7168, I = 2048
        {"name": "product swiglu decode", "op": "product", "n": 24, "N": 2048, "K": 7168, "bias": False,
         "act": "swiglu", "res": False, "out": "bf16", "scale": 1.0},
        # the output head over a large vocabulary of odd size, fp32 logits for a batch of 16 decoded tokens
        {"name": "product head", "op": "product", "n": 16, "N": 100003, "K": 4096, "bias": False, "act": "none",
         "res": False, "out": "f32", "scale": 1.0},
        # a ragged chunk of a prompt, H = 2880, bias and residual
        {"name": "product ragged chunk", "op": "product", "n": 333, "N": 2880, "K": 2880, "bias": True, "act": "none",
         "res": True, "out": "bf16", "scale": 1.0},
        # the output projection of long prompts with the residual scaled in: bound by the matrix units
        {"name": "product prompts", "op": "product", "n": 4096, "N": 7168, "K": 7168, "bias": False, "act": "none",
         "res": True, "out": "bf16", "scale": 0.22},
        # one conversation, the usual settings (temperature 1, top-k 64, top-p 0.95), fp32 logits: latency
        {"name": "sample one row", "op": "sample", "n": 1, "V": 100003, "elem": "f32", "mode": "usual"},
        # a decode batch whose requests all have settings of their own, bf16 logits of odd rows
        {"name": "sample decode batch", "op": "sample", "n": 48, "V": 100003, "elem": "bf16", "mode": "mixed"},
        # many rows of a wide vocabulary by top-p alone, which has to weigh all of it
        {"name": "sample many rows", "op": "sample", "n": 160, "V": 200003, "elem": "f32", "mode": "top-p"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "product", "product", "sample", "sample"])
    if op == "norm":
        if rng.random() < 0.3:
            return {"op": op, "n": _spread(rng, 1, 4000), "heads": _spread(rng, 1, 64), "dim": 8 * _spread(rng, 4, 32),
                    "res": "", "post": "", "pre": rng.choice(["rms", "rms1", "layer"]), "gate": rng.choice(["", "head"]),
                    "scale": 1.0}
        post = rng.choice(["", "rms", "rms1", "layer"])
        return {"op": op, "n": _spread(rng, 1, 4000), "heads": 0, "dim": 8 * _spread(rng, 32, 1024),
                "res": rng.choice(["bf16", "f32"]), "post": post, "pre": rng.choice(["rms", "rms1", "layer"]),
                "gate": rng.choice(["", "token", "column", "silu"]), "scale": rng.choice([1.0, 0.5, 0.22])}
    if op == "product":
        K = 8 * _spread(rng, 16, 1024)
        act = rng.choice(["none", "none", "sigmoid", "silu", "gelu", "swiglu"])
        N = _spread(rng, 16, 20000)
        n = _spread(rng, 1, max(1, min(4096, 80_000_000_000 // (N * K * (2 if act == "swiglu" else 1)))))
        return {"op": op, "n": n, "N": N, "K": K, "bias": rng.random() < 0.5, "act": act, "res": rng.random() < 0.5,
                "out": rng.choice(["bf16", "bf16", "f32"]), "scale": rng.choice([1.0, 0.5])}
    return {"op": op, "n": _spread(rng, 1, 128), "V": _spread(rng, 300, 200000), "elem": rng.choice(["bf16", "f32"]),
            "mode": rng.choice(["usual", "mixed", "mixed", "top-p", "min-p", "all"])}


def work(case):
    op, n = case["op"], case["n"]
    if op == "norm":
        values, D = n * max(1, case["heads"]) * case["dim"], case["dim"]
        size = {"": 0, "bf16": 4, "f32": 8}[case["res"]]
        gate = {"": 0, "token": 2 * n, "head": 2 * n * case["heads"], "column": 2 * D, "silu": 2 * values}[case["gate"]]
        rows = sum({"": 0, "rms": 2, "rms1": 2, "layer": 4}[case[k]] * D for k in ("post", "pre"))
        return {"bytes": values * (4 + size) + gate + rows, "flops": values * (4 + 5 * (case["post"] != ""))}
    if op == "product":
        N, K = case["N"], case["K"]
        rows, out = N * (2 if case["act"] == "swiglu" else 1), 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (rows * K + n * K + rows * case["bias"]) + n * N * out * (1 + case["res"]), "flops": 2 * n * rows * K}
    return {"bytes": n * (case["V"] * (2 if case["elem"] == "bf16" else 4) + 28), "flops": 4 * n * case["V"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, device=DEV, generator=g) * std


def _norm_state(case, g):
    n, D = case["n"], case["dim"]
    shape = (n, case["heads"], D) if case["heads"] else (n, D)
    s = {"x": _normal(g, *shape).bfloat16(), "y": torch.empty(shape, dtype=torch.bfloat16, device=DEV)}
    if case["res"]:
        kind = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        # a residual stream has grown over the layers, and a few of its columns more than the others
        r = _normal(g, *shape, std=4.0)
        r[..., ::509] *= 30.0
        s["res"], s["res_out"] = r.to(kind), torch.empty(shape, dtype=kind, device=DEV)
    for k in ("post", "pre"):
        if case[k]:
            s[k + "_w"] = (_normal(g, D, std=0.2) + (0.0 if case[k] == "rms1" else 1.0)).bfloat16()
        if case[k] == "layer":
            s[k + "_b"] = _normal(g, D, std=0.1).bfloat16()
    if case["gate"]:
        size = {"token": (n, 1), "head": (*shape[:-1], 1), "column": (D,), "silu": shape}[case["gate"]]
        s["gate"] = _normal(g, *size).bfloat16()
    return s


def _product_state(case, g):
    n, N, K = case["n"], case["N"], case["K"]
    rows, kind = N * (2 if case["act"] == "swiglu" else 1), torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s = {"x": _normal(g, n, K).bfloat16(), "w": _normal(g, rows, K, std=0.02).bfloat16(),
         "y": torch.empty(n, N, dtype=kind, device=DEV)}
    if case["bias"]:
        s["bias"] = _normal(g, rows, std=0.1).bfloat16()
    if case["res"]:
        s["res"] = _normal(g, n, N, std=4.0).to(kind)
    return s


def _settings(mode, n, rng):
    """(temperature, top-k, top-p, min-p) of every row."""
    if mode == "usual":
        return [(1.0, 64, 0.95, 0.0)] * n
    if mode == "top-p":
        return [(rng.choice([0.7, 1.0]), 0, rng.choice([0.9, 0.95, 0.99]), 0.0) for _ in range(n)]
    if mode == "min-p":
        return [(rng.choice([1.0, 1.5]), 0, 1.0, rng.choice([0.02, 0.05, 0.1])) for _ in range(n)]
    if mode == "all":
        return [(rng.choice([0.8, 1.0, 1.3]), 0, 1.0, 0.0) for _ in range(n)]
    return [(rng.choice([0.0, 0.3, 0.6, 0.8, 1.0, 1.0, 1.3]), rng.choice([0, 1, 20, 50, 64, 500, 3000]),
             rng.choice([1.0, 0.5, 0.8, 0.9, 0.95, 0.95]), rng.choice([0.0, 0.0, 0.0, 0.05, 0.1])) for _ in range(n)]


def _sample_state(case, g, seed):
    n, V = case["n"], case["V"]
    logits = _normal(g, n, V, std=2.0)
    # a few hundred words go with the context, more or less surely; a grammar forbids some words
    some = min(V, 400)
    at = torch.randint(0, V, (n, some), device=DEV, generator=g)
    lift = 9.0 + 3.0 * torch.rand(n, 1, device=DEV, generator=g)
    logits.scatter_add_(1, at, lift * torch.rand(n, some, device=DEV, generator=g))
    logits[:, 7::1013] = -math.inf
    logits = logits.bfloat16() if case["elem"] == "bf16" else logits
    rows = _settings(case["mode"], n, random.Random(int(seed) * 31 + 7))
    t, k, p, m = zip(*rows)
    return {"logits": logits, "u": torch.rand(n, device=DEV, generator=g),
            "temperature": torch.tensor(t, dtype=torch.float32, device=DEV),
            "top_k": torch.tensor(k, dtype=torch.int32, device=DEV),
            "top_p": torch.tensor(p, dtype=torch.float32, device=DEV),
            "min_p": torch.tensor(m, dtype=torch.float32, device=DEV),
            "ids": torch.empty(n, dtype=torch.int32, device=DEV),
            "logprob": torch.empty(n, dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = _norm_state(case, g) if op == "norm" else _product_state(case, g) if op == "product" else _sample_state(case, g, seed)
    s["case"] = case
    if own:
        import offloaded_expert_slot_amd as oes
        s["oes"] = oes
        if op == "norm":
            for k in ("post", "pre"):
                if case[k]:
                    s[k] = oes.Norm(s[k + "_w"], bias=s.get(k + "_b"), kind="layer" if case[k] == "layer" else "rms",
                                    eps=EPS, offset=1.0 if case[k] == "rms1" else 0.0)
        if op == "sample":
            s["ws"] = torch.empty(oes.sample_workspace_bytes(case["n"], case["V"]), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    v = v * (w.float() + 1.0 if kind == "rms1" else w.float())
    return v + b.float() if kind == "layer" else v


def _plain_norm(case, s):
    v = s["x"].float()
    if case["post"]:
        v = _normed(v, case["post"], s["post_w"], s.get("post_b"))
    if case["gate"]:
        gate = s["gate"].float()
        v = v * (gate / (1.0 + torch.exp(-gate)) if case["gate"] == "silu" else 1.0 / (1.0 + torch.exp(-gate)))
    v = v * case["scale"]
    if case["res"]:
        # the next norm is that of the residual as the stream holds it
        s["res_out"].copy_(s["res"].float() + v)
        v = s["res_out"].float()
    s["y"].copy_(_normed(v, case["pre"], s["pre_w"], s.get("pre_b")))
    return _norm_outputs(case, s)


def _norm_outputs(case, s):
    return {"res": s["res_out"], "y": s["y"]} if case["res"] else {"y": s["y"]}


def _plain_product(case, s):
    z = s["x"].float() @ s["w"].float().t()
    if case["bias"]:
        z = z + s["bias"].float()
    N, act = case["N"], case["act"]
    if act == "swiglu":
        z = z[:, :N] / (1.0 + torch.exp(-z[:, :N])) * z[:, N:]
    elif act == "sigmoid":
        z = 1.0 / (1.0 + torch.exp(-z))
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif act == "gelu":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    z = z * case["scale"]
    s["y"].copy_(s["res"].float() + z if case["res"] else z)
    return s["y"]


def _plain_sample(case, s):
    n, V = case["n"], case["V"]
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"].double())[:, None]
    # the largest first, equal ones by index: a stable descending sort
    logits, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    z = logits.double() / t
    w = torch.exp(z - z[:, :1])
    rank = torch.arange(V, device=DEV)
    k = torch.where(s["top_k"] > 0, s["top_k"], V)
    keep = rank < torch.where(greedy, 1, k)[:, None]
    before = torch.cumsum(w * keep, -1)
    total = before[:, -1:].clone()
    before = before - w * keep
    p = s["top_p"].double()[:, None]
    keep &= (before < p * total) | (p >= 1.0)
    keep &= w >= s["min_p"].double()[:, None]
    # the running sum in the order of the vocabulary
    kept = torch.zeros_like(w).scatter_(1, order, w * keep)
    running = torch.cumsum(kept, -1)
    total = running[:, -1:]
    ids = (running <= s["u"].double()[:, None] * total).sum(-1)
    s["ids"].copy_(ids)
    weight = kept.gather(1, ids.clamp(max=V - 1)[:, None])
    s["logprob"].copy_(torch.log(weight / total)[:, 0])
    return {"ids": s["ids"], "logprob": s["logprob"]}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "product": _plain_product, "sample": _plain_sample}[op](case, s)
    oes = s["oes"]
    if op == "norm":
        gate = s.get("gate")
        oes.norm(s["x"], s["y"], pre=s["pre"], post=s.get("post"), gate=gate,
                 gate_act="silu" if case["gate"] == "silu" else "sigmoid", scale=case["scale"], res=s.get("res"),
                 res_out=s.get("res_out"))
        return _norm_outputs(case, s)
    if op == "product":
        oes.linear_bf16(s["x"], s["w"], s["y"], bias=s.get("bias"), act=case["act"], scale=case["scale"], res=s.get("res"))
        return s["y"]
    oes.sample(s["logits"], s["u"], s["ids"], s["ws"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
               min_p=s["min_p"], logprob=s["logprob"])
    return {"ids": s["ids"], "logprob": s["logprob"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_normed(v, kind, w, b):
    w = w.double()
    if kind == "rms1":
        w = w + 1
    if kind != "layer":
        return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS) * w
    var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
    return (v - mean) / torch.sqrt(var + EPS) * w + b.double()


def _exact_norm(case, s):
    v = s["x"].double()
    if case["post"]:
        v = _exact_normed(v, case["post"], s["post_w"], s.get("post_b"))
    if case["gate"]:
        gate = s["gate"].double()
        v = v * torch.sigmoid(gate) * (gate if case["gate"] == "silu" else 1)
    v = v * case["scale"]
    got = {}
    if case["res"]:
        got["res"] = s["res"].double() + v
        v = got["res"].to(s["res"].dtype).double()
    got["y"] = _exact_normed(v, case["pre"], s["pre_w"], s.get("pre_b"))
    return got


def _exact_product(case, s):
    n, N, act = case["n"], case["N"], case["act"]
    x, y = s["x"].double(), torch.empty(n, N, dtype=torch.float64, device=DEV)

    def part(r, e):
        z = torch.mm(x, s["w"][r:e].double().t().contiguous())
        return z + s["bias"][r:e].double() if case["bias"] else z

    for r in range(0, N, 8192):
        e = min(N, r + 8192)
        z = part(r, e)
        if act in ("swiglu", "silu"):
            gate = z * torch.sigmoid(z)
            z = gate * part(N + r, N + e) if act == "swiglu" else gate
        elif act == "sigmoid":
            z = torch.sigmoid(z)
        elif act == "gelu":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * z * (1 + 0.044715 * z * z))
        y[:, r:e] = z * case["scale"]
    return y + s["res"].double() if case["res"] else y


def _exact_sample(case, s):
    """The log-probabilities alone, row by row: a token is a whole number and has to be the same."""
    logits = s["logits"].float().cpu().numpy()
    values = [s[k].cpu().numpy().astype(np.float64) for k in ("temperature", "top_k", "top_p", "min_p", "u")]
    out = np.empty(case["n"])
    for i in range(case["n"]):
        t, k, p, m, u = (v[i] for v in values)
        if t <= 0:
            out[i] = 0.0
            continue
        row = logits[i].astype(np.float64)
        order = np.lexsort((np.arange(row.size), -row))
        order = order[:int(k)] if k > 0 else order
        w = np.exp((row[order] - row[order[0]]) / t)
        if p < 1:
            order = order[:1 + np.searchsorted(np.cumsum(w), p * w.sum())]
        w = np.exp((row - row[order[0]]) / t)
        order = np.sort(order[w[order] >= m])
        sums = np.cumsum(w[order])
        token = order[np.searchsorted(sums, u * sums[-1], side="right")]
        out[i] = (row[token] - row.max()) / t - math.log(sums[-1])
    return {"ids": None, "logprob": torch.from_numpy(out).to(DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "sample": _exact_sample}[case["op"]](case, s)

"""The attention half of a decoder layer around the expert step: cases, plain forms and 64-bit values.

Operators, and what a pass of each computes:

  linear   y = x . W^T for 4-bit weights W with group scales, in the 4-bit bank formats of the expert banks
  rope     rotary positions on q and k, with k and v written into the pages of the cache
  attn     attention of each sequence's new tokens over its paged cache, and the log-sum-exp of every row
  weigh    the attention weight that every cache entry receives, added to what it had
  evict    the entries with the largest accumulated weight kept (with the first and the last ones), the rest
           dropped and the cache closed up in place

``run`` computes the plain forms in float32 (angles in float64), or calls the library where ``own`` is true.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the fused q, k, v projection of one decoded token, H = 2048: a few microseconds, latency
        {"name": "linear q4_0 one token", "op": "linear", "fmt": "q4_0", "n": 1, "N": 5120, "K": 2048},
        # the output head over a large vocabulary of odd size, H = 7168, for a batch of 16 decoded tokens
        {"name": "linear nvfp4 head", "op": "linear", "fmt": "nvfp4", "n": 16, "N": 100003, "K": 7168},
        # a decode batch at positions far into a long context, bf16 cache
        {"name": "rope decode", "op": "rope", "batch": 32, "q_len": 1, "lens": 11, "max_len": 4096, "heads": 32,
         "kv_heads": 4, "dim": 128, "rot": 128, "layout": "half", "scaling": "none", "elem": "bf16", "page": 16,
         "far": 120000},
        # ragged prompts, half of each head rotated in the interleaved layout, positions scaled, e4m3 cache
        {"name": "rope prompts", "op": "rope", "batch": 4, "q_len": 3000, "lens": 12, "max_len": 4096, "heads": 64,
         "kv_heads": 8, "dim": 128, "rot": 64, "layout": "interleaved", "scaling": "yarn", "elem": "e4m3",
         "page": 64, "far": 0},
        # one decoded token early in a conversation: the smallest call
        {"name": "attn one token", "op": "attn", "batch": 1, "q_len": 1, "lens": 21, "max_len": 600, "heads": 32,
         "kv_heads": 4, "dim": 128, "elem": "bf16", "page": 16, "window": 0, "spare": 0},
        # a decode batch of contexts of all lengths up to 16 k, e4m3 cache
        {"name": "attn decode batch", "op": "attn", "batch": 32, "q_len": 1, "lens": 22, "max_len": 16384,
         "heads": 32, "kv_heads": 4, "dim": 128, "elem": "e4m3", "page": 64, "window": 0, "spare": 0},
        # short ragged chunks of several requests with a sliding window, 64-wide heads, spare rows at the end
        {"name": "attn ragged window", "op": "attn", "batch": 6, "q_len": 700, "lens": 23, "max_len": 4001,
         "heads": 64, "kv_heads": 8, "dim": 64, "elem": "bf16", "page": 32, "window": 128, "spare": 5},
        # one chunk of a long prompt behind 22 k cached entries: the largest, bound by the matrix units
        {"name": "attn long chunk", "op": "attn", "batch": 1, "q_len": 2048, "lens": 24, "max_len": 24111,
         "heads": 32, "kv_heads": 4, "dim": 128, "elem": "bf16", "page": 16, "window": 0, "spare": 0},
        # the weights of one decode step
        {"name": "weigh decode", "op": "weigh", "batch": 16, "q_len": 1, "lens": 31, "max_len": 8192, "heads": 32,
         "kv_heads": 4, "dim": 128, "elem": "bf16", "page": 16, "window": 0, "spare": 0},
        # the weights of ragged prompt chunks, 64-wide heads, e4m3 cache
        {"name": "weigh chunks", "op": "weigh", "batch": 3, "q_len": 1000, "lens": 32, "max_len": 8111, "heads": 64,
         "kv_heads": 8, "dim": 64, "elem": "e4m3", "page": 64, "window": 0, "spare": 0},
        # a decode batch that makes room every 32 steps
        {"name": "evict every 32 steps", "op": "evict", "batch": 16, "lens": 41, "min_len": 2080, "max_len": 2080,
         "kv_heads": 4, "dim": 128, "elem": "bf16", "page": 16, "budget": 2048, "first": 4, "last": 64},
        # after long prompts: caches cut down to a quarter
        {"name": "evict after prompts", "op": "evict", "batch": 4, "lens": 42, "min_len": 9000, "max_len": 16384,
         "kv_heads": 8, "dim": 128, "elem": "bf16", "page": 64, "budget": 4099, "first": 4, "last": 512},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "attn", "attn", "attn", "weigh", "evict"])
    if op == "linear":
        K = 32 * _spread(rng, 8, 224)
        N = _spread(rng, 64, 100000)
        return {"op": op, "fmt": rng.choice(["q4_0", "nvfp4", "mxfp4_t"]), "n": _spread(rng, 1, 64), "N": N, "K": K}
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = {"op": op, "lens": rng.randrange(1 << 20), "kv_heads": kv_heads, "dim": dim,
         "elem": rng.choice(["bf16", "e4m3"]), "page": rng.choice([16, 32, 64])}
    if op == "evict":
        most = _spread(rng, 64, 16384)
        budget = _spread(rng, 16, most)
        return {**c, "batch": _spread(rng, 1, 16), "min_len": 1 + most // 2, "max_len": most, "budget": budget,
                "first": rng.randint(0, min(4, budget // 4)), "last": rng.randint(0, budget // 2)}
    c["heads"] = kv_heads * rng.choice([1, 4, 6, 8])
    if op == "rope":
        return {**c, "batch": _spread(rng, 1, 16), "q_len": _spread(rng, 1, 1000), "max_len": _spread(rng, 1000, 5000),
                "rot": 2 * rng.randint(8, dim // 2), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "far": rng.choice([0, 30000, 500000])}
    if rng.random() < 0.5:  # decode steps
        batch, q_len, most = _spread(rng, 1, 32), rng.choice([1, 1, 1, 2, 4]), _spread(rng, 16, 16000)
    else:  # chunks of prompts
        batch, q_len, most = _spread(rng, 1, 6), _spread(rng, 8, 1000), _spread(rng, 1000, 8000)
    return {**c, "batch": batch, "q_len": q_len, "max_len": most, "window": rng.choice([0, 0, 0, 100, 1024]),
            "spare": rng.choice([0, 0, 3])}


def _lens(case):
    """(new tokens, cache entries with them) of every sequence of a case."""
    rng = random.Random(case["lens"])
    B = case["batch"]
    if case["op"] == "evict":
        return [0] * B, [rng.randint(case["min_len"], case["max_len"]) for _ in range(B)]
    q = [case["q_len"] if b == 0 or case["q_len"] < 5 else rng.randint(1, case["q_len"]) for b in range(B)]
    # the first sequence has the full length; the others' are spread over the logarithm
    lens = [max(case["max_len"] if b == 0 else _spread(rng, 1, case["max_len"]), q[b]) for b in range(B)]
    return q, lens


def _seen(q, n, window):
    """Cache entries that the q last of n tokens see together (each its predecessors, itself and no more than window)."""
    if not window:
        return q * (n - q) + q * (q + 1) // 2
    return sum(min(n - q + i + 1, window) for i in range(q))


def work(case):
    op = case["op"]
    if op == "linear":
        group, extra = {"q4_0": (32, 0), "nvfp4": (16, 2), "mxfp4_t": (32, 2)}[case["fmt"]]
        N, K, n = case["N"], case["K"], case["n"]
        scale = 2 if case["fmt"] == "q4_0" else 1
        return {"bytes": N * (K // 2 + K // group * scale + extra) + 2 * n * (K + N), "flops": 2 * n * N * K}
    q, lens = _lens(case)
    B, D, Hkv = case["batch"], case["dim"], case["kv_heads"]
    size = 2 if case["elem"] == "bf16" else 1
    if op == "evict":
        # only what stands behind the first dropped entry moves: of e dropped at random among n, it stands at n / (e + 1)
        keep = case["budget"]
        moved = int(sum(max(0.0, keep - n / (n - keep + 1)) for n in lens if n > keep)) * Hkv
        return {"bytes": 4 * sum(lens) * Hkv + moved * (2 * 2 * D * size + 4) + 4 * B * Hkv * keep, "flops": sum(lens) * Hkv}
    Hq, n = case["heads"], sum(q)
    if op == "rope":
        return {"bytes": n * (2 * Hq * D * 2 + 2 * Hkv * D * (2 + size) + 4), "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    w = case["window"]
    entries = sum(min(n_, q_ - 1 + w) if w else n_ for q_, n_ in zip(q, lens))
    pairs = sum(_seen(q_, n_, w) for q_, n_ in zip(q, lens))
    if op == "attn":
        return {"bytes": 2 * entries * Hkv * D * size + n * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}
    return {"bytes": entries * Hkv * (D * size + 8) + n * Hq * (2 * D + 4), "flops": 2 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, device=DEV, generator=g) * std


def _linear_state(case, g):
    n, N, K, fmt = case["n"], case["N"], case["K"], case["fmt"]
    s = {"x": _normal(g, n, K).bfloat16(), "y": torch.empty(n, N, dtype=torch.bfloat16, device=DEV)}
    # codes as quantised N(0, 0.02) weights have them: every code occurs; scales about 0.02 / 3
    if fmt == "mxfp4_t":
        codes = torch.randint(0, 256, (K // 32, N, 16), dtype=torch.uint8, device=DEV, generator=g)
        scale = torch.randint(117, 121, (K // 32, N), dtype=torch.uint8, device=DEV, generator=g)
        s["banks"] = [codes, scale, _normal(g, N, std=0.02).bfloat16()]
    else:
        codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        if fmt == "q4_0":
            s["banks"] = [codes, (0.002 + 0.006 * torch.rand(N, K // 32, device=DEV, generator=g)).half()]
        else:
            scale = torch.randint(0x48, 0x7f, (N, K // 16), dtype=torch.uint8, device=DEV, generator=g)
            s["banks"] = [codes, scale, (2e-5 + 4e-5 * torch.rand(N, device=DEV, generator=g)).half()]
    return s


def _pages(case, g, lens, spare=3):
    """Scattered pages of the cache, with the tables of the sequences: used pages in random order, some free ones."""
    ps, Hkv, D = case["page"], case["kv_heads"], case["dim"]
    used = [-(-n // ps) for n in lens]
    cols = max(1, max(used))
    num = sum(used) + spare
    order = torch.randperm(num, device=DEV, generator=g).int()
    table = torch.zeros(len(lens), cols, dtype=torch.int32)
    at = 0
    order = order.cpu()
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    k = _normal(g, num, ps, Hkv, D)
    v = _normal(g, num, ps, Hkv, D)
    s = {"table": table.to(DEV), "len": torch.tensor(lens, dtype=torch.int32, device=DEV), "k_scale": 1.0,
         "v_scale": 1.0}
    if case["elem"] == "e4m3":
        s["k_scale"], s["v_scale"] = 0.02, 0.0125
        k = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    return {**s, "k": k, "v": v}


def _starts(q):
    at = [0]
    for n in q:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "linear":
        s = _linear_state(case, g)
    else:
        q, lens = _lens(case)
        s = _pages(case, g, lens)
        Hkv, D, ps = case["kv_heads"], case["dim"], case["page"]
        cap = s["table"].shape[1] * ps
        if op == "evict":
            B = case["batch"]
            # accumulated weights: most entries have next to none, a few have much
            s["acc"] = _normal(g, B, Hkv, cap).mul_(2.5).exp_()
            s["kept"] = torch.empty(B, Hkv, case["budget"], dtype=torch.int32, device=DEV)
            s["new_len"] = torch.empty(B, dtype=torch.int32, device=DEV)
        else:
            Hq, n = case["heads"], sum(q)
            rows = n + case.get("spare", 0)
            s["q_start"] = _starts(q)
            s["q"] = _normal(g, rows, Hq, D).bfloat16()
        if op == "rope":
            s["k_new"], s["v_new"] = _normal(g, n, Hkv, D).bfloat16(), _normal(g, n, Hkv, D).bfloat16()
            s["q_out"] = torch.empty_like(s["q"])
            pos = [case["far"] + m - a + i for a, m in zip(q, lens) for i in range(a)]
            s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
            freq, s["mscale"] = _frequencies(case)
            s["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        if op in ("attn", "weigh"):
            s["scale"] = 1.0 / math.sqrt(D)
            s["lse"] = torch.zeros(rows, Hq, dtype=torch.float32, device=DEV)
            s["out"] = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV)
        if op == "weigh":
            _plain_attn(case, s)  # the log-sum-exps as the attention of the same step left them
            del s["out"]
            s["acc"] = 0.01 * torch.rand(case["batch"], Hkv, cap, device=DEV, generator=g)
    s["case"] = case
    if own:
        import offloaded_expert_slot_amd as oes
        s["oes"] = oes
        if op != "linear":
            s["kv"] = oes.KvPages(s["k"], s["v"], s["table"], s["len"], s["k_scale"], s["v_scale"])
        if op == "attn":
            need = oes.attn_workspace_bytes(s["kv"], case["heads"], s["q"].shape[0])
            s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
        if op == "evict":
            need = oes.kv_evict_workspace_bytes(s["kv"], case["budget"])
            s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    return s


def _frequencies(case):
    """Angle per position of every rotated pair (radians), and the factor on the rotated values."""
    rot, base, factor, trained = case["rot"], 10000.0, 8.0, 4096
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "ntk":
        wide = base * factor ** (rot / (rot - 2.0))
        return [wide ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if case["scaling"] == "yarn":
        def at(turns):  # the (fractional) pair that makes so many turns over the trained length
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(at(32.0))), min(rot - 1.0, math.ceil(at(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ------------------------------------------------------------------ plain forms
def _values(codes, scale):
    return codes.float() * scale if codes.dtype == torch.float8_e4m3fn else codes.float()


def _plain_linear(case, s):
    x, banks, fmt, N, K = s["x"].float(), s["banks"], case["fmt"], case["N"], case["K"]
    codes = banks[0]
    lo, hi = codes & 15, codes >> 4
    if fmt == "q4_0":  # byte j of a block of 16: element j in the low nibble, element j + 16 in the high one
        both = torch.cat([lo.view(N, K // 32, 16), hi.view(N, K // 32, 16)], dim=2)
        w = (both.float() - 8.0) * banks[1].float()[:, :, None]
    else:
        lut = torch.tensor(E2M1, device=DEV)
        both = lut[torch.stack([lo, hi], dim=-1).int()]
        if fmt == "nvfp4":
            scale = banks[1].view(torch.float8_e4m3fn).float() * banks[2].float()[:, None]
            w = both.view(N, K // 16, 16) * scale[:, :, None]
        else:
            w = both.view(K // 32, N, 32) * torch.exp2(banks[1].float() - 127.0)[:, :, None]
            w = w.permute(1, 0, 2)
    y = x @ w.reshape(N, K).t().contiguous()
    if fmt == "mxfp4_t":
        y = y + banks[2].float()
    s["y"].copy_(y)
    return s["y"]


def _entry_index(table, ps, count):
    """Flat (page, place) index of entries 0 .. count - 1 of every sequence: [B, count]."""
    j = torch.arange(count, device=DEV)
    return table[:, j // ps].long() * ps + j % ps


def _plain_rope(case, s):
    rot, mscale = case["rot"], s["mscale"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (angle.cos() * mscale).float()[:, None, :], (angle.sin() * mscale).float()[:, None, :]

    def turned(x):
        x = x.float()
        head, rest = x[..., :rot], x[..., rot:]
        if case["layout"] == "half":
            a, b = head[..., :rot // 2], head[..., rot // 2:]
            return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
        a, b = head[..., 0::2], head[..., 1::2]
        both = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        return torch.cat([both, rest], dim=-1)

    s["q_out"].copy_(turned(s["q"]))
    start, ps = s["q_start"].long(), case["page"]
    token = torch.arange(s["pos"].numel(), device=DEV)
    seq = torch.searchsorted(start, token, right=True) - 1
    entry = s["len"].long()[seq] - (start[seq + 1] - start[seq]) + token - start[seq]
    page = s["table"][seq, entry // ps].long()
    for name, new, scale in (("k", turned(s["k_new"]), s["k_scale"]), ("v", s["v_new"].float(), s["v_scale"])):
        if case["elem"] == "e4m3":
            new = (new / scale).clamp(-448, 448)
        s[name][page, entry % ps] = new.to(s[name].dtype)
    return _rope_outputs(case, s)


def _rope_outputs(case, s):
    # e4m3 values are bf16 numbers, so the caches come back as the values that they hold
    return {"q": s["q_out"], "k": s["k"].bfloat16(), "v": s["v"].bfloat16()}


def _padded(case, s):
    """Scores of the new tokens padded to the longest: [B, Hkv, Qmax * G, L], -inf where masked; and their places."""
    start, lens = s["q_start"].long(), s["len"].long()
    qs, ls = _lens(case)
    B, Hkv, G, D = len(qs), case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    Q, L = max(qs), max(ls)
    i, j = torch.arange(Q, device=DEV), torch.arange(L, device=DEV)
    q_len = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    live = i < q_len[:, None]
    flat = _entry_index(s["table"], case["page"], L)
    k = _values(s["k"].flatten(0, 1)[flat], s["k_scale"])
    q = s["q"][row].float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    at = (lens - q_len)[:, None] + i  # the entry of each new token
    see = (j <= at[:, :, None]) & (j < lens[:, None, None]) & live[:, :, None]
    if case["window"]:
        see &= j > at[:, :, None] - case["window"]
    see = see[:, None, :, None, :].expand(B, 1, Q, G, L).reshape(B, 1, Q * G, L)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(s["scale"])
    return scores.masked_fill_(~see, -math.inf), flat, row, live


def _unpadded(x, row, live, B, Hkv, G):
    """[B, Hkv, Q * G, ...] back to the packed rows: ([rows, Hq, ...], which rows)."""
    Q = row.shape[1]
    x = x.view(B, Hkv, Q, G, *x.shape[3:]).transpose(1, 2).flatten(2, 3)
    return x[live], row[live]


def _plain_attn(case, s):
    B, Hkv = case["batch"], case["kv_heads"]
    G = case["heads"] // Hkv
    scores, flat, row, live = _padded(case, s)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(s["v"].flatten(0, 1)[flat], s["v_scale"])
    out = torch.matmul(p, v.transpose(1, 2).contiguous()) / total.clamp(min=1e-30)
    lse = (total.log() + top).squeeze(-1)
    out, at = _unpadded(out, row, live, B, Hkv, G)
    s["out"][at] = out.to(s["out"].dtype)
    s["lse"][at] = _unpadded(lse, row, live, B, Hkv, G)[0]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weigh(case, s):
    B, Hkv = case["batch"], case["kv_heads"]
    G = case["heads"] // Hkv
    scores, _, row, live = _padded(case, s)
    lse = s["lse"][row].view(B, row.shape[1], Hkv, G).transpose(1, 2).reshape(B, Hkv, -1, 1)
    weight = scores.sub_(lse).exp_().sum(2)
    s["acc"][:, :, :weight.shape[2]] += weight
    return s["acc"]


def _plain_evict(case, s):
    B, Hkv, ps = case["batch"], case["kv_heads"], case["page"]
    budget, cap = case["budget"], s["acc"].shape[2]
    lens = s["len"].long()
    n = lens[:, None, None]
    j = torch.arange(cap, device=DEV)
    keep_always = (j < case["first"]) | ((j >= n - case["last"]) & (j < n))
    key = torch.where(keep_always, math.inf, s["acc"])
    key = torch.where(j < n, key, -math.inf)
    # the largest first, equal ones by index: a stable descending sort; the kept ones back in their order
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    full = torch.sort(order, dim=-1).values
    if cap < budget:
        full = torch.nn.functional.pad(full, (0, budget - cap))
    slot = torch.arange(budget, device=DEV)
    new_len = torch.minimum(lens, torch.full_like(lens, budget))
    live = (slot < new_len[:, None])[:, None, :].expand(B, Hkv, budget)
    full = torch.where((lens > budget)[:, None, None], full, slot.expand(B, Hkv, budget))
    s["kept"].copy_(torch.where(live, full, -1))
    s["new_len"].copy_(new_len)
    b, h, i = live.nonzero(as_tuple=True)
    src = full[b, h, i]
    page, place = s["table"][b, i // ps].long(), i % ps
    page_from, place_from = s["table"][b, src // ps].long(), src % ps
    for name in ("k", "v"):
        raw = s[name].view(torch.int16 if s[name].dtype == torch.bfloat16 else torch.uint8)
        raw[page, place, h] = raw[page_from, place_from, h]
    s["acc"][b, h, i] = s["acc"][b, h, src]
    return _evict_outputs(s)


def _evict_outputs(s):
    return {"kept": s["kept"], "len": s["new_len"], "acc": s["acc"], "k": s["k"].bfloat16(), "v": s["v"].bfloat16()}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"linear": _plain_linear, "rope": _plain_rope, "attn": _plain_attn, "weigh": _plain_weigh,
                "evict": _plain_evict}[op](case, s)
    oes = s["oes"]
    if op == "linear":
        oes.linear(case["fmt"], s["x"], s["banks"], s["y"])
        return s["y"]
    kv = s["kv"]
    if op == "rope":
        oes.rope_append(s["q"], s["q_out"], s["k_new"], s["v_new"], s["freq"], s["pos"], kv, s["q_start"],
                        layout=case["layout"], mscale=s["mscale"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]} if case["elem"] == "bf16" else _rope_outputs(case, s)
    if op == "attn":
        oes.attn(s["q"], s["out"], kv, s["q_start"], s["scale"], s["ws"], window=case["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weigh":
        oes.attn_weigh(s["q"], s["lse"], kv, s["q_start"], s["scale"], s["acc"], window=case["window"])
        return s["acc"]
    oes.kv_evict(kv, s["acc"], case["budget"], s["kept"], s["new_len"], s["ws"], first=case["first"],
                 last=case["last"])
    return {"kept": s["kept"], "len": s["new_len"], "acc": s["acc"], "k": s["k"], "v": s["v"]} \
        if case["elem"] == "bf16" else _evict_outputs(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3_value(u):
    """Value of e4m3 bytes from their fields."""
    u = u.long()
    e, m = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    return torch.where(u >= 128, -mag, mag)


def _to_e4m3(x):
    """The nearest e4m3 value (ties to even), up to 448."""
    x = x.clamp(-448, 448)
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _stored(case, s, name):
    if case["elem"] == "e4m3":
        return _e4m3_value(s[name].view(torch.uint8)) * s[name + "_scale"]
    return s[name].double()


def _of_sequence(case, s, stored, b, count):
    """Entries 0 .. count - 1 of sequence b, [count, Hkv, D]."""
    ps = case["page"]
    pages = stored[s["table"][b, :-(-count // ps)].long()]
    return pages.reshape(-1, *pages.shape[2:])[:count]


def _exact_linear(case, s):
    N, K, fmt = case["N"], case["K"], case["fmt"]
    x, y = s["x"].double(), torch.empty(case["n"], N, dtype=torch.float64, device=DEV)
    for r in range(0, N, 16384):
        e = min(N, r + 16384)
        w = torch.empty(e - r, K, dtype=torch.float64, device=DEV)
        if fmt == "q4_0":
            c = s["banks"][0][r:e].long().view(e - r, K // 32, 16)
            blocks = w.view(e - r, K // 32, 32)
            blocks[..., :16], blocks[..., 16:] = c % 16 - 8, c // 16 - 8
            blocks *= s["banks"][1][r:e].double()[..., None]
        else:
            c = s["banks"][0][r:e] if fmt == "nvfp4" else s["banks"][0][:, r:e].transpose(0, 1).reshape(e - r, K // 2)
            for part, code in ((0, c.long() % 16), (1, c.long() // 16)):
                exp, man = (code >> 1) & 3, (code & 1).double()
                mag = torch.where(exp > 0, (1 + man / 2) * torch.exp2(exp.double() - 1), man / 2)
                w[:, part::2] = torch.where(code >= 8, -mag, mag)
            if fmt == "nvfp4":
                w.view(e - r, K // 16, 16).mul_(_e4m3_value(s["banks"][1][r:e])[..., None])
                w *= s["banks"][2][r:e].double()[:, None]
            else:
                w.view(e - r, K // 32, 32).mul_(torch.exp2(s["banks"][1][:, r:e].t().double() - 127)[..., None])
        y[:, r:e] = x @ w.t().contiguous()
    return y + s["banks"][2].double() if fmt == "mxfp4_t" else y


def _exact_rope(case, s):
    rot, half = case["rot"], case["rot"] // 2
    first = torch.arange(half, device=DEV) * (1 if case["layout"] == "half" else 2)
    second = first + (half if case["layout"] == "half" else 1)
    turn = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(s["pos"].numel(), half),
                       s["pos"].double()[:, None] * s["freq"])[:, None, :]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    got = {"q": turned(s["q"])}
    q, lens = _lens(case)
    for name, new in (("k", turned(s["k_new"])), ("v", s["v_new"].double())):
        if case["elem"] == "e4m3":
            new, held = _to_e4m3(new / s[name + "_scale"]), _e4m3_value(s[name].view(torch.uint8))
        else:
            held = s[name].double()
        at = 0
        for b, (a, m) in enumerate(zip(q, lens)):
            j = torch.arange(m - a, m, device=DEV)
            held[s["table"][b, j // case["page"]].long(), j % case["page"]] = new[at:at + a]
            at += a
        got[name] = held
    return got


def _exact_scores(case, s, keys, b, h, first, a, m):
    """Masked scores [a, G, m] of sequence b's new tokens against head h's entries."""
    G = case["heads"] // case["kv_heads"]
    q = s["q"][first:first + a, h * G:(h + 1) * G].double()
    scores = (q.reshape(a * G, -1) @ keys[:, h].t().contiguous()).view(a, G, m) * s["scale"]
    i, j = torch.arange(a, device=DEV)[:, None, None], torch.arange(m, device=DEV)
    hidden = j > m - a + i
    if case["window"]:
        hidden = hidden | (m - a + i - j >= case["window"])
    return scores.masked_fill_(hidden, -math.inf)


def _exact_attn(case, s):
    G = case["heads"] // case["kv_heads"]
    out, lse = s["out"].double(), s["lse"].double()
    k, v = _stored(case, s, "k"), _stored(case, s, "v")
    first = 0
    for b, (a, m) in enumerate(zip(*_lens(case))):
        keys, values = _of_sequence(case, s, k, b, m), _of_sequence(case, s, v, b, m)
        for h in range(case["kv_heads"]):
            scores = _exact_scores(case, s, keys, b, h, first, a, m)
            total = torch.logsumexp(scores, -1)
            p = torch.exp_(scores.sub_(total[..., None])).view(a * G, m)
            out[first:first + a, h * G:(h + 1) * G] = (p @ values[:, h].contiguous()).view(a, G, -1)
            lse[first:first + a, h * G:(h + 1) * G] = total
        first += a
    return {"out": out, "lse": lse}


def _exact_weigh(case, s):
    G = case["heads"] // case["kv_heads"]
    acc, k, first = s["acc"].double(), _stored(case, s, "k"), 0
    for b, (a, m) in enumerate(zip(*_lens(case))):
        keys = _of_sequence(case, s, k, b, m)
        for h in range(case["kv_heads"]):
            scores = _exact_scores(case, s, keys, b, h, first, a, m)
            total = s["lse"][first:first + a, h * G:(h + 1) * G].double()
            acc[b, h, :m] += torch.exp_(scores.sub_(total[..., None])).sum((0, 1))
        first += a
    return acc


def _exact_evict(case, s):
    acc, k, v = s["acc"].double(), s["k"].double(), s["v"].double()
    ps = case["page"]
    for b, m in enumerate(_lens(case)[1]):
        if m <= case["budget"]:
            continue
        for h in range(case["kv_heads"]):
            j = list(range(m))
            always = set(j[:case["first"]]) | set(j[m - case["last"]:])
            w = acc[b, h, :m].tolist()
            ranked = sorted((x for x in j if x not in always), key=lambda x: (-w[x], x))
            kept = torch.tensor(sorted(always | set(ranked[:case["budget"] - len(always)])), device=DEV)
            to = torch.arange(case["budget"], device=DEV)
            for held in (k, v):
                held[s["table"][b, to // ps].long(), to % ps, h] = \
                    held[s["table"][b, kept // ps].long(), kept % ps, h].clone()
            acc[b, h, to] = acc[b, h, kept].clone()
    return {"kept": None, "len": None, "acc": acc, "k": k, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "attn": _exact_attn, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](case, s)

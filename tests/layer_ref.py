"""Plain float64 references of the operators around the expert step (not a test module).

Everything runs on the CPU in double precision, one sequence and head at a time, from
the definitions; nothing here is shared with the kernels.
"""
import math

import torch

U = 2.0 ** -24            # half a step of fp32
BF = 2.0 ** -8            # half a step of bf16


def e2m1(codes):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    return table[codes.long()]


def nibbles(codes):
    """[..., bytes] -> [..., 2 * bytes], low nibble first."""
    return torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)


def weights(fmt, banks, N, K):
    """[N, K] float64 weights of a bank format (without the mxfp4_t bias)."""
    w0, w1 = banks[0].cpu(), banks[1].cpu()
    if fmt == "q4_0":
        c = w0.view(N, K // 32, 16).long()
        q = torch.cat([c & 15, c >> 4], dim=2).double() - 8
        return (q * w1.double().view(N, K // 32, 1)).view(N, K)
    if fmt == "nvfp4":
        s = w1.view(torch.float8_e4m3fn).to(torch.float32).double().view(N, K // 16, 1)
        return (e2m1(nibbles(w0.view(N, K // 2))).view(N, K // 16, 16) * s).view(N, K) * banks[2].cpu().double()[:, None]
    e = w1.view(torch.uint8).view(K // 32, N, 1).double()
    s = torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))
    return (e2m1(nibbles(w0.view(K // 32, N, 16))) * s).permute(1, 0, 2).reshape(N, K)


def linear(fmt, x, banks, N):
    """(y, bound): the product in float64, and how far a correct kernel's bf16 may be from it.

    bound = half a bf16 step of y, plus fp32 rounding: every product and sum is off by at
    most U of the magnitudes that it adds, over at most 40 + K / 32 additions that a
    product goes through; for q4_0 the kernels may count a code as 128 + q and take
    136 * sum(x) off again, which makes the magnitudes within a block of 32 up to
    (143 + 136) |x| for its 33 additions.
    """
    K = x.shape[1]
    xd, w = x.cpu().double(), weights(fmt, banks, N, K)
    y = xd @ w.t()
    mag = xd.abs() @ w.abs().t()
    err = (40 + K / 32) * U * mag
    if fmt == "q4_0":
        d = banks[1].cpu().double().view(N, K // 32).abs()
        err = err + 33 * 279 * U * (xd.abs().view(-1, K // 32, 32).sum(2) @ d.t())
    if fmt == "mxfp4_t" and banks[2] is not None:
        y = y + banks[2].cpu().double()
    return y, BF * (y.abs() + err) + err + 1e-38


def turn(x, pos, freq, mscale, layout, rot):
    """Rotary positions in float64."""
    x = x.cpu().double().clone()
    half = rot // 2
    i0 = torch.arange(half) if layout == "half" else 2 * torch.arange(half)
    i1 = i0 + half if layout == "half" else i0 + 1
    angle = pos.cpu().double()[:, None] * freq.cpu()
    c, s = (mscale * angle.cos())[:, None], (mscale * angle.sin())[:, None]
    a, b = x[..., i0].clone(), x[..., i1].clone()
    x[..., i0], x[..., i1] = a * c - b * s, a * s + b * c
    return x


def to_e4m3(x):
    """Nearest e4m3 value (ties to even) of clamped x, from the format's spacing."""
    x = x.clamp(-448, 448)
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


class Cache:
    """A paged cache with every sequence's pages scattered, and its plain copy."""

    def __init__(self, seed, lens, kv_heads, dim, page, elem="bf16", head_major=False, spare=2, device="cuda:0",
                 cols=None, fill=None):
        g = torch.Generator().manual_seed(seed)
        used = [-(-max(0, n) // page) for n in lens]
        self.cols = cols or max([1] + used)
        self.pages = sum(used) + spare
        order = torch.randperm(self.pages, generator=g).int()
        self.table = torch.zeros(len(lens), self.cols, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        shape = (self.pages, kv_heads, page, dim) if head_major else (self.pages, page, kv_heads, dim)
        self.k, self.v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        if fill is not None:  # what no sequence holds
            live = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    live[self.table[b, j // page], j % page] = True
            dead = ~live[:, None, :, None] if head_major else ~live[:, :, None, None]
            self.k, self.v = self.k.masked_fill(dead, fill), self.v.masked_fill(dead, fill)
        self.k_scale = self.v_scale = 1.0
        if elem == "e4m3":
            self.k_scale, self.v_scale = 0.02, 0.0125
            self.k = (self.k / self.k_scale).to(torch.float8_e4m3fn)
            self.v = (self.v / self.v_scale).to(torch.float8_e4m3fn)
        else:
            self.k, self.v = self.k.bfloat16(), self.v.bfloat16()
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.page, self.lens, self.elem, self.kv_heads, self.dim = page, list(lens), elem, kv_heads, dim
        if device:
            self.to(device)

    def to(self, device):
        self.dk, self.dv = self.k.to(device), self.v.to(device)
        self.dtable, self.dlen = self.table.to(device), torch.tensor(self.lens, dtype=torch.int32, device=device)
        return self

    def handle(self, oes):
        return oes.KvPages(self.dk, self.dv, self.dtable, self.dlen, self.k_scale, self.v_scale)

    def entries(self, b):
        """(k, v) float64 [len, kv_heads, dim] of sequence b, and which of its entries have a page."""
        j = torch.arange(max(0, self.lens[b]))
        p = self.table[b, j // self.page].long()
        ok = (p >= 0) & (p < self.pages)
        p = p.clamp(0, self.pages - 1)
        k = self.k.to(torch.float32)[p, j % self.page].double() * self.k_scale
        v = self.v.to(torch.float32)[p, j % self.page].double() * self.v_scale
        return k, v, ok


def attention(q, cache, q_start, scale, window=0):
    """(out, lse, bound, p): float64 attention; bound on a bf16 result; p[b]: [q_len, Hq, len] weights.

    bound: half a bf16 step of the result; the probabilities are rounded to bf16 (half a step
    each, in sum at most BF of sum p |v|); a score is off by at most (D + 4) U of
    scale sum |q k| plus 4 U of itself, a probability by e times as much, relatively,
    where e^x - 1 <= 2 x; the sums over the entries by (n / 16 + 64) U of sum p |v|: n / 16
    chained steps of matrix products and at most 64 joins.
    """
    n, Hq, D = q.shape
    G = Hq // cache.kv_heads
    out, lse, bound = torch.zeros(n, Hq, D).double(), torch.full((n, Hq), -math.inf).double(), torch.zeros(n, Hq, D).double()
    probs = []
    for b in range(len(cache.lens)):
        first, last = q_start[b], q_start[b + 1]
        a, m = last - first, max(0, cache.lens[b])
        if a == 0 or m == 0:
            probs.append(torch.zeros(a, Hq, m).double())
            continue
        k, v, ok = cache.entries(b)
        at = torch.arange(a)[:, None] + m - a
        j = torch.arange(m)
        see = (j <= at) & ok
        if window:
            see &= j > at - window
        p_all = torch.zeros(a, Hq, m).double()
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            qq = q[first:last, h].cpu().double()
            s = (qq @ kk.t() * scale).masked_fill(~see, -math.inf)
            mag = (qq.abs() @ kk.abs().t() * scale).nan_to_num(0, 0, 0).masked_fill(~see, 0).amax(1, keepdim=True)
            top = s.amax(1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            e = torch.exp(s - top)
            total = e.sum(1, keepdim=True)
            p = torch.where(see & (total > 0), e / total.clamp(min=1e-300), torch.zeros_like(e))
            vz = torch.where(see.any(0)[:, None], vv, torch.zeros_like(vv))
            p_all[:, h] = p
            out[first:last, h] = p @ vz
            lse[first:last, h] = torch.where(total > 0, top + total.clamp(min=1e-300).log(), torch.full_like(top, -math.inf))[:, 0]
            spread = p @ vz.abs()
            rel = 2 * ((D + 4) * U * mag + 4 * U * s.masked_fill(~see, 0).abs().amax(1, keepdim=True)) * 2
            bound[first:last, h] = BF * out[first:last, h].abs() + (BF + rel + (m / 16 + 64) * U) * spread * (1 + BF) + 1e-30
        probs.append(p_all)
    return out, lse, bound, probs


def evict(acc, lens, cache, budget, first, last):
    """kept [B, H, budget] (-1 filled), by sorting (weight descending, index ascending)."""
    B, H = len(lens), cache.kv_heads
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    for b, m in enumerate(lens):
        for h in range(H):
            if m <= budget:
                kept[b, h, :m] = torch.arange(m, dtype=torch.int32)
                continue
            always = set(range(first)) | set(range(m - last, m))
            w = acc[b, h, :m].tolist()
            key = lambda x: (w[x] != w[x], -w[x] if w[x] == w[x] else 0.0, x)  # noqa: E731  NaN last
            ranked = sorted((x for x in range(m) if x not in always), key=key)
            kept[b, h] = torch.tensor(sorted(always | set(ranked[:budget - len(always)])), dtype=torch.int32)
    return kept

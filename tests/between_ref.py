"""Plain float64 references of the operators between the blocks, with the bounds that a correct
fp32 kernel keeps (not a test module).  Everything runs on the CPU, from the definitions."""
import math
from fractions import Fraction

import numpy as np
import torch

U = 2.0 ** -24            # half a step of fp32
BF = 2.0 ** -8            # half a step of bf16


def stored(y, err, kind):
    """Bound of a value rounded once to `kind`, whose unrounded form is off by at most err."""
    return (BF if kind == torch.bfloat16 else U) * (y.abs() + err) + err + 1e-38


# ------------------------------------------------------------------ norm
def normed(v, err, spec):
    """(norm of rows v, bound): v is known up to err.

    Every sum over the row goes through at most 40 + dim / 64 additions of fp32 (a thread's own
    values, then a tree), each off by U of the magnitudes added; so a mean is off by at most
    c mean|v|, the mean square by a share 2 c of itself (and what err does to it), the root by
    half of that, and five more roundings make the value.
    """
    if spec is None:
        return v, err
    D = v.shape[-1]
    c = (40 + D / 64) * U
    d, off = v, err
    if spec["kind"] == "layer":
        d = v - v.mean(-1, keepdim=True)
        off = err + (c * v.abs() + err).mean(-1, keepdim=True) + U * d.abs()
    ms = d.square().mean(-1, keepdim=True)
    inv = 1 / torch.sqrt(ms + spec["eps"])
    ms_off = (2 * d.abs() * off + off * off).mean(-1, keepdim=True) + 2 * c * ms
    share = ms_off / (ms + spec["eps"]).clamp(min=1e-300)   # of inv: half of it to first order
    gain = torch.ones(D, dtype=torch.float64)
    if spec["w"] is not None:
        gain = spec["offset"] + spec["w"].cpu().double()
    b = torch.zeros(D, dtype=torch.float64) if spec["b"] is None else spec["b"].cpu().double()
    y = d * inv * gain + b
    mag = (d * inv * gain).abs()
    return y, gain.abs() * inv * off * (1 + share) + mag * (share + 5 * U) + U * (mag + b.abs())


def gate_of(g, act):
    """(value, share by which fp32 is off): exp of a rounded argument is off by |g| U, and a few steps more."""
    if act == "plain":
        return g, torch.zeros_like(g)
    s = torch.sigmoid(g)
    return (s if act == "sigmoid" else g * s), (g.abs() + 8) * 4 * U


def norm(x, post, gate, act, scale, res):
    """(r, bound of r before it is rounded)."""
    v = x.cpu().double()
    v, err = normed(v, torch.zeros_like(v), post)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    if gate is not None:
        g, share = gate_of(gate.cpu().double().expand(v.shape), act)
        err = g.abs() * (err * (1 + share) + v.abs() * share)
        v = v * g
    v, err = v * scale, abs(scale) * err + 3 * U * (v * scale).abs()
    if res is not None:
        v = v + res.cpu().double()
        err = err + U * (v.abs() + err)
    return v, err


# ------------------------------------------------------------------ product
def product(x, w, bias, act, scale, res):
    """(y, bound before y is rounded): a product goes through at most 48 + K / 32 additions."""
    xd, wd = x.cpu().double(), w.cpu().double()
    z = xd @ wd.t()
    err = (48 + xd.shape[1] / 32) * U * (xd.abs() @ wd.abs().t())
    if bias is not None:
        z = z + bias.cpu().double()
        err = err + U * (z.abs() + err)
    if act == "swiglu":
        N = w.shape[0] // 2
        (g, u), (eg, eu) = (z[:, :N], z[:, N:]), (err[:, :N], err[:, N:])
        s = g * torch.sigmoid(g)
        es = 1.1 * eg + s.abs() * (g.abs() + 8) * 4 * U
        a, ea = s * u, es * u.abs() + s.abs() * eu + es * eu
        ea = ea + U * a.abs()
    elif act == "sigmoid":
        a = torch.sigmoid(z)
        ea = 0.25 * err + a * (z.abs() + 8) * 4 * U
    elif act == "silu":
        a = z * torch.sigmoid(z)
        ea = 1.1 * err + a.abs() * (z.abs() + 8) * 4 * U
    elif act == "gelu":
        t = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        a = 0.5 * z * (1 + torch.tanh(t))
        # tanh is off by steps of 1; its argument by 4 steps, where it matters as long as |t| < 20
        ea = 1.2 * err + z.abs() * 4 * U + a.abs() * (t.abs().clamp(max=20) + 8) * 8 * U
    else:
        a, ea = z, err
    scale = float(torch.tensor(scale, dtype=torch.float32))
    y, ey = a * scale, abs(scale) * ea + U * (a * scale).abs()
    if res is not None:
        y = y + res.cpu().double()
        ey = ey + U * (y.abs() + ey)
    return y, ey


# ------------------------------------------------------------------ sample
def sample_row(row, t, k, p, m, u):
    """(token, logprob, margin) of one row by the definition, in float64 and exact fractions of its sums.

    margin: how near a decision of the float64 form came to its border, as a share of the sum: a
    kernel that weighs to 2^-40 or better decides alike where it is larger than that.  Exact
    ties (weights of 1 alone) are decided exactly and count as no margin.
    """
    row = np.asarray(row, dtype=np.float64)
    valid = ~(np.isnan(row) | (row == -np.inf))
    if not valid.any():
        return -1, -np.inf, 1.0
    safe = np.where(valid, row, -np.inf)
    order = np.lexsort((np.arange(row.size), -safe))[:int(valid.sum())]
    top = row[order[0]]
    if not t > 0:
        return int(order[0]), 0.0, 1.0
    if top == np.inf:
        w = (row[order] == np.inf).astype(np.float64)
    else:
        w = np.exp((row[order] - top) / float(t))
    w[w < 2.0 ** -44] = 0.0
    margin = 1.0
    exact = bool(np.isin(w, (0.0, 1.0)).all())
    if k > 0:
        order, w = order[:k], w[:k]
    if p < 1:
        sums = np.cumsum(w)
        if exact:
            want = Fraction(float(p)) * int(sums[-1])
            last = next(i for i, s in enumerate(sums) if int(s) >= want)
        else:
            want = float(p) * sums[-1]
            last = int(np.searchsorted(sums, want)) if p > 0 else 0
            if p > 0:
                margin = min(margin, float(np.abs(sums - want).min() / sums[-1]))
        order, w = order[:last + 1], w[:last + 1]
    if m > 0:
        least = min(float(m), 1.0)
        margin = margin if exact else min(margin, float(np.where(w == 1.0, 1.0, np.abs(w - least)).min()))
        order, w = order[w >= least], w[w >= least]
    by = np.argsort(order)
    order, w = order[by], w[by]
    sums = np.cumsum(w)
    total = sums[-1]
    u = 0.0 if not u >= 0 else float(u)
    if u >= 1:
        at = int(np.nonzero(w)[0][-1])
    elif exact:
        want = Fraction(u) * int(total)
        at = next(i for i, s in enumerate(sums) if int(s) > want)
    else:
        at = int(np.searchsorted(sums, u * total, side="right"))
        if u > 0:
            margin = min(margin, float(np.abs(sums - u * total).min() / total))
    token = int(order[at])
    lp = (0.0 if top == np.inf else (row[token] - top) / float(t)) - math.log(total)
    return token, lp, margin

"""The operators between the blocks on the GPU, against float64 references: every type, kind and
broadcast, ragged and odd sizes, strides, in place, values that are not finite, masked rows, ties,
repeats, graphs, other streams, and a decode step of all of them together."""
import math

import numpy as np
import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import between_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g) * std


def _within(got, ref, bound, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


# ------------------------------------------------------------------ norm
def _spec(g, kind, dim, dtype, offset=0.0, weight=True, bias=None, eps=1e-6):
    if kind is None:
        return None, None
    w = (_randn(g, dim, std=0.3) + 1 - offset).to(dtype) if weight else None
    bias = kind == "layer" if bias is None else bias
    b = _randn(g, dim, std=0.2).to(dtype) if bias else None
    own = oes.Norm(None if w is None else w.to(DEV), None if b is None else b.to(DEV), kind=kind, eps=eps, offset=offset)
    return own, {"kind": kind, "w": w, "b": b, "offset": offset, "eps": eps}


def _padded(t, extra, fill=None):
    """t on the GPU as a view whose rows (and heads) are `extra` values further apart, and the whole."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), 7.0, dtype=t.dtype, device=DEV)
    view = wide[..., :t.shape[-1]]
    if fill is not False:
        view.copy_(t)
    return view, wide


def _check_norm(x, pre=None, post=None, gate=None, act="plain", scale=1.0, res=None, store=True, y=True, extra=0, inplace=""):
    (pre, pre_r), (post, post_r) = pre or (None, None), post or (None, None)
    kind = None if res is None else res.dtype
    r, err = R.norm(x, post_r, gate, act, scale, res)
    xv, _ = _padded(x, extra)
    rv = None if res is None else _padded(res, extra)[0]
    gv = None if gate is None else gate.to(DEV)
    ov = ow = yv = yw = None
    if store:
        kind = kind or BF16
        ov, ow = (rv, None) if "res" in inplace else _padded(torch.empty(x.shape, dtype=kind), extra, False)
    if y:
        yv, yw = (xv, None) if "y" in inplace else _padded(torch.empty(x.shape, dtype=BF16), extra, False)
    oes.norm(xv, yv, pre=pre, post=post, gate=gv, gate_act=act, scale=scale, res=rv, res_out=ov)
    if store:
        _within(ov, r, R.stored(r, err, kind), "r")
        if ow is not None and extra:
            assert (ow[..., x.shape[-1]:] == 7).all(), "written behind a row"
        r, err = ov.double().cpu(), torch.zeros_like(r)
    if y:
        want, err = R.normed(r, err, pre_r)
        _within(yv, want, R.stored(want, err, BF16), "y")
        if yw is not None and extra:
            assert (yw[..., x.shape[-1]:] == 7).all(), "written behind a row"


DIMS = [8, 16, 24, 56, 64, 72, 128, 200, 256, 504, 512, 520, 768, 1024, 1032, 2040, 2048, 2056, 2880, 4096, 4104, 7168, 8192,
        8200, 12296, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_sums(dim, kind):
    g = _gen(dim)
    x, res = _randn(g, 3, dim).bfloat16(), _randn(g, 3, dim, std=3.0).bfloat16()
    _check_norm(x, pre=_spec(g, kind, dim, BF16), res=res, extra=8)
    _check_norm(x, pre=_spec(g, kind, dim, F32, bias=True), res=res.float(), extra=16, scale=-0.3)
    _check_norm(x, pre=_spec(g, kind, dim, BF16), post=_spec(g, kind, dim, F32, offset=1.0), res=res)


@pytest.mark.parametrize("dim", [8, 40, 64, 128, 264, 1024, 2880, 5120])
@pytest.mark.parametrize("gate", ["row", "head", "column", "all", "one"])
@pytest.mark.parametrize("act", ["plain", "sigmoid", "silu"])
def test_norm_gates(dim, gate, act):
    g = _gen(dim + len(gate))
    x = _randn(g, 5, 3, dim).bfloat16()
    shape = {"row": (5, 1, 1), "head": (5, 3, 1), "column": (dim,), "all": (5, 3, dim), "one": (1,)}[gate]
    gt = _randn(g, *shape, std=2.0).bfloat16()
    _check_norm(x, pre=_spec(g, "rms", dim, BF16), gate=gt, act=act, store=False)
    _check_norm(x, post=_spec(g, "rms", dim, BF16), gate=gt, act=act, scale=0.22, res=_randn(g, 5, 3, dim), extra=8)


@pytest.mark.parametrize("n,heads,dim", [(1, 1, 64), (1, 32, 128), (7, 5, 64), (33, 4, 40), (300, 2, 128), (5, 1, 512),
                                         (2, 3, 2056), (4097, 1, 64), (1030, 1, 2048), (600, 1, 4096), (2100, 1, 8192)])
def test_norm_of_many_rows(n, heads, dim):
    g = _gen(n)
    x = _randn(g, n, heads, dim).bfloat16()
    _check_norm(x, pre=_spec(g, "rms", dim, BF16), store=False, extra=8)
    _check_norm(x, pre=_spec(g, "layer", dim, BF16), res=_randn(g, n, heads, dim))
    _check_norm(x, pre=_spec(g, "rms", dim, BF16, offset=1.0), store=False, inplace="y")


@pytest.mark.parametrize("dim", [64, 2048, 7168])
@pytest.mark.parametrize("x32", [False, True])
def test_norm_parts_left_out(dim, x32):
    g = _gen(dim)
    x, res = _randn(g, 4, dim), _randn(g, 4, dim, std=2.0)
    x = x if x32 else x.bfloat16()
    pre, post = _spec(g, "rms", dim, BF16), _spec(g, "layer", dim, F32)
    _check_norm(x)                                          # r = x
    _check_norm(x, y=False, res=res)                        # the sum alone
    _check_norm(x, y=False, post=post, res=res.bfloat16(), inplace="res")
    _check_norm(x, store=False, res=res, pre=pre)           # the norm of a sum that is not kept
    _check_norm(x, store=False, post=post, pre=pre)
    _check_norm(x, pre=_spec(g, "rms", dim, BF16, weight=False, eps=0.1), res=res, inplace="res")
    _check_norm(x, pre=_spec(g, "layer", dim, BF16, weight=False, bias=True), store=False)
    if not x32:
        _check_norm(x, pre=pre, post=post, res=res, inplace="res y")


@pytest.mark.parametrize("dim", [64, 1024, 8200])
def test_norm_extremes(dim):
    """NaN and infinity stay in their rows; zeros, tiny rows, and rows of one large value."""
    g = _gen(dim)
    x = _randn(g, 8, dim).bfloat16()
    x[1, 3], x[2, dim - 1], x[3] = math.nan, math.inf, 0.0
    x[4] = 2.0 ** -60
    x[5, 1:], x[5, 0] = 0.0, 2.0 ** 60
    x[6] = 2.0 ** 100          # squares beyond fp32: the norm is 0
    own, spec = _spec(g, "rms", dim, BF16)
    y = torch.empty(8, dim, dtype=BF16, device=DEV)
    oes.norm(x.to(DEV), y, pre=own)
    y = y.cpu()
    assert y[1].isnan().all()
    assert y[2, dim - 1].isnan() and (y[2, :-1] == 0).all()
    assert (y[6] == 0).all()
    rows = [0, 3, 4, 5, 7]
    want, err = R.normed(x[rows].double(), torch.zeros(len(rows), dim, dtype=torch.float64), spec)
    _within(y[rows], want, R.stored(want, err, BF16), "rows")


def test_norm_layer_of_rows_far_from_zero():
    """The mean is taken off before the squares: a large common value does not drown the variance."""
    dim, g = 2048, _gen(3)
    x = (1000.0 + _randn(g, 4, dim)).float()
    _check_norm(x, pre=_spec(g, "layer", dim, F32), store=False)


# ------------------------------------------------------------------ product
def _check_product(n, N, K, act="none", bias=False, res=False, out=BF16, scale=1.0, inplace=False, pad=0, seed=0, wpad=0):
    g = _gen(n * 7 + N * 3 + K + seed)
    rows = 2 * N if act == "swiglu" else N
    x, w = _randn(g, n, K).bfloat16(), _randn(g, rows, K, std=2.0 / math.sqrt(K)).bfloat16()
    b = _randn(g, rows).bfloat16() if bias else None
    r = _randn(g, n, N, std=2.0).to(out) if res else None
    xv, wv = _padded(x, 8 if pad else 0)[0], _padded(w, wpad)[0]
    yv, yw = _padded(torch.empty(n, N, dtype=out), pad, False)
    rv = None if r is None else _padded(r, pad)[0]
    if inplace:
        yv.copy_(rv)
        rv = yv
    guard = torch.full((n + 1, N), 7.0, dtype=out, device=DEV)
    oes.linear_bf16(xv, wv, yv, bias=None if b is None else b.to(DEV), act=act, scale=scale, res=rv)
    y, err = R.product(x, w, b, act, scale, r)
    what = (n, N, K, act, bias, res, out, pad)
    _within(yv, y, R.stored(y, err, out), what)
    if pad:
        assert (yw[:, N:] == 7).all(), "written behind a row"
    if not inplace:   # rows behind the last one
        oes.linear_bf16(xv, wv, guard[:n], bias=None if b is None else b.to(DEV), act=act, scale=scale, res=rv)
        assert (guard[n] == 7).all(), "written behind the last row"
        assert torch.equal(guard[:n], yv), "two calls differ"


@pytest.mark.parametrize("n,N,K", [(1, 1, 8), (1, 1, 2048), (1, 7, 16), (1, 515, 2048), (1, 64, 7168), (1, 2048, 24), (2, 33, 160),
                                   (3, 1030, 256), (4, 16, 72), (5, 16, 1024), (8, 100, 2880), (9, 17, 4104), (15, 47, 416),
                                   (16, 256, 512), (17, 129, 128), (24, 2000, 1000), (31, 513, 520), (32, 80, 544),
                                   (33, 80, 544), (48, 300, 2056), (64, 31, 2048), (65, 200, 192), (100, 2880, 328),
                                   (127, 127, 136), (128, 128, 64), (129, 257, 200), (200, 48, 64), (257, 511, 776),
                                   (300, 1000, 2880), (513, 769, 264), (1000, 130, 1544)])
def test_product(n, N, K):
    _check_product(n, N, K, pad=3)
    _check_product(n, N, K, act="swiglu", bias=True, scale=0.5)
    _check_product(n, N, K, bias=True, res=True, out=F32, pad=1, wpad=8)
    _check_product(n, N, K, act="silu", res=True, scale=-1.5, inplace=True)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("n", [1, 20, 130])
def test_product_epilogues(act, out, n):
    for bias in (False, True):
        for res in (False, True):
            _check_product(n, 150, 320, act=act, bias=bias, res=res, out=out, scale=0.75 if res else 1.0, pad=2 * bias)


@pytest.mark.parametrize("n,N,K,act", [(1, 20011, 512, "none"), (16, 30001, 256, "none"), (40, 25003, 264, "swiglu"),
                                       (520, 4099, 136, "silu"), (2100, 1030, 72, "none"), (700, 3001, 1032, "swiglu"),
                                       (1, 9000, 4096, "swiglu"), (64, 6000, 1024, "gelu"), (4097, 260, 64, "none")])
def test_product_many_rows(n, N, K, act):
    _check_product(n, N, K, act=act, pad=1)
    _check_product(n, N, K, act=act, bias=True, res=True, out=F32)


@pytest.mark.parametrize("n", [1, 3, 16, 40, 150, 600])
def test_product_extremes(n):
    """NaN and infinity of x reach their own rows, of W their own columns; large and tiny values."""
    N, K, g = 300, 520, _gen(n)
    x, w = _randn(g, n, K).bfloat16(), _randn(g, N, K, std=0.05).bfloat16()
    clean = torch.empty(n, N, dtype=F32, device=DEV)
    oes.linear_bf16(x.to(DEV), w.to(DEV), clean)
    x[0, K - 1], w[5, 0], w[N - 1, K - 1] = math.nan, math.inf, math.nan
    y = torch.empty(n, N, dtype=F32, device=DEV)
    oes.linear_bf16(x.to(DEV), w.to(DEV), y)
    assert y[0].isnan().all()
    keep = [c for c in range(N) if c not in (5, N - 1)]
    assert torch.equal(y[1:][:, keep], clean[1:][:, keep])
    assert not y[:, 5].isfinite().any() and y[:, N - 1].isnan().all()
    big = torch.full((n, K), 2.0 ** 60, dtype=BF16, device=DEV)
    tiny = torch.full((N, K), 2.0 ** -60, dtype=BF16, device=DEV)
    oes.linear_bf16(big, tiny, y)
    assert (y == K).all()


def test_product_of_rows_far_apart():
    """Rows of W more than 2^31 elements apart in all."""
    N, K, stride = 40, 64, 1 << 26
    g = _gen(11)
    whole = torch.empty(stride * (N - 1) + K, dtype=BF16, device=DEV)
    w = whole.as_strided((N, K), (stride, 1))
    ref = _randn(g, N, K).bfloat16()
    w.copy_(ref)
    for n in (2, 70, 300):
        x = _randn(g, n, K).bfloat16()
        y = torch.empty(n, N, dtype=F32, device=DEV)
        oes.linear_bf16(x.to(DEV), w, y)
        want, err = R.product(x, ref, None, "none", 1.0, None)
        _within(y, want, R.stored(want, err, F32), n)


# ------------------------------------------------------------------ sample
def _sample(logits, u, t=None, k=None, p=None, m=None, **over):
    n = logits.shape[0]

    def dev(v, dtype):
        return None if v is None else torch.as_tensor(v, dtype=dtype).expand(n).contiguous().to(DEV)

    ids = torch.full((n + 1,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((n + 1,), 7.0, device=DEV)
    ws = torch.randint(0, 256, (max(16, oes.sample_workspace_bytes(n, logits.shape[1])),), dtype=torch.uint8, device=DEV)
    oes.sample(logits if logits.is_cuda else logits.to(DEV), dev(u, F32), ids[:n], ws, temperature=dev(t, F32),
               top_k=dev(k, torch.int32), top_p=dev(p, F32), min_p=dev(m, F32), logprob=lp[:n], **over)
    assert ids[n] == -7 and lp[n] == 7
    return ids[:n].cpu(), lp[:n].cpu()


def _check_sample(logits, u, t=None, k=None, p=None, m=None):
    """Every row against the definition; rows whose decision is within 2^-36 of a border may not occur."""
    n = logits.shape[0]
    ids, lp = _sample(logits, u, t, k, p, m)

    def at(v, i, default, dtype=F32):
        return default if v is None else torch.as_tensor(v, dtype=dtype).expand(n)[i].item()

    rows = logits.float().cpu().numpy()
    for i in range(n):
        args = at(t, i, 1.0), at(k, i, 0, torch.int32), at(p, i, 1.0), at(m, i, 0.0), at(u, i, 0.0)
        token, want, margin = R.sample_row(rows[i], *args)
        assert margin > 2.0 ** -36, ("the inputs leave the choice open", i, args)
        assert ids[i] == token, (i, args, int(ids[i]), token)
        if want == -math.inf:
            assert lp[i] == -math.inf
        else:
            # the weights are off by 2^-44 each; the result is rounded to fp32 once
            assert abs(lp[i].item() - want) <= 2.0 ** -24 * abs(want) + 1e-7 * 2.0 ** -4 + 1e-30, (i, args, lp[i].item(), want)


def _logits(g, n, V, dtype):
    """As a model has them: most near one another, some hundred far above."""
    l = _randn(g, n, V, std=2.0)
    some = max(1, min(V // 3, 300))
    at = torch.randint(0, V, (n, some), generator=g)
    l.scatter_add_(1, at, 10 * torch.rand(n, some, generator=g))
    return l.to(dtype)


SETTINGS = [(1.0, 0, 1.0, 0.0), (1.0, 64, 0.95, 0.0), (0.7, 0, 0.9, 0.0), (1.0, 0, 0.999, 0.0), (1.3, 20, 1.0, 0.0),
            (1.0, 0, 1.0, 0.05), (0.5, 500, 0.8, 0.02), (0.0, 5, 0.5, 0.1), (-1.0, 0, 1.0, 0.0), (math.nan, 3, 0.9, 0.0),
            (1.0, 1, 1.0, 0.0), (1.0, 1 << 30, 0.6, 0.0), (2.0, 3000, 0.99, 0.001), (1.0, -5, 2.0, -1.0),
            (1.0, 0, 1e-6, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, -1.0, 2.0), (1.0, 0, math.nan, math.nan), (0.05, 0, 0.9, 0.0),
            (100.0, 0, 0.5, 0.0), (1e-30, 0, 1.0, 0.0), (math.inf, 7, 1.0, 0.0), (1.0, 0, 1.0, 1.0), (8.0, 0, 0.97, 0.0)]


@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 65, 255, 1000, 1025, 4097, 20011, 50257, 100003, 262147])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample(V, dtype):
    g = _gen(V)
    n = len(SETTINGS)
    t, k, p, m = (list(v) for v in zip(*SETTINGS))
    for u in (torch.rand(n, generator=g), torch.rand(n, generator=g)):
        _check_sample(_logits(g, n, V, dtype), u, t, k, p, m)


@pytest.mark.parametrize("n", [1, 2, 5, 17, 100, 300])
def test_sample_rows(n):
    g = _gen(n)
    logits = _logits(g, n, 5003, F32)
    u = torch.rand(n, generator=g)
    _check_sample(logits, u, 1.0, 64, 0.95)
    _check_sample(logits, u)
    _check_sample(logits, u, 0.8, None, 0.9, 0.01)


@pytest.mark.parametrize("V", [1, 100, 9001, 70001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_masks(V, dtype):
    """-inf, NaN, +inf and the type's lowest value in places and in whole rows."""
    g, lowest = _gen(V), torch.finfo(dtype).min
    rows = []
    for fill in (-math.inf, math.nan, lowest):
        r = _logits(g, 4, V, dtype)
        r[0] = fill
        r[1, ::2] = fill
        r[2, 1:] = fill
        r[3, :-1] = fill
        rows.append(r)
    r = _logits(g, 4, V, dtype)
    r[0, V // 2] = math.inf
    r[1, ::3] = math.inf
    r[2] = math.inf
    r[3] = math.nan
    r[3, V - 1] = math.inf
    logits = torch.cat(rows + [r])
    n = logits.shape[0]
    u = torch.rand(n, generator=g)
    for s in ((None, None, None, None), (1.0, 5, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (0.7, 0, 0.5, 0.1), (1.0, 70000, 1.0, 0.0)):
        _check_sample(logits, u, *s)


@pytest.mark.parametrize("V", [8, 1000, 40000, 131072])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_ties(V, dtype):
    """Equal logits go by index, in every rule and by exact fractions of their number."""
    u = [0.0, 0.125, 0.5, 0.75, 1 - 2.0 ** -24, 1.0, 2.0, math.nan, -1.0]
    n = len(u)
    flat = torch.full((n, V), 3.25, dtype=dtype)
    for s in ((None, None, None, None), (1.0, 5, 1.0, 0.0), (0.5, 0, 0.5, 0.0), (2.0, V // 2, 0.25, 1.0), (1.0, V - 1, 0.75, 0.5)):
        _check_sample(flat, u, *s)
    steps = torch.arange(V).remainder(7).float().expand(n, V).to(dtype)     # seven values, many times each
    _check_sample(steps, [0.03 + 0.1 * i for i in range(n)], 1.0, V // 7 + 3, 0.9)
    two = torch.zeros(n, V, dtype=dtype)
    two[:, 1::2] = -0.0                                                       # zeros of both signs are equal
    _check_sample(two, u, 1.0, V // 2 + 1, 0.5)


def test_sample_follows_the_weights():
    """Over a grid of numbers every token comes up as often as its share says."""
    g, n, V = _gen(5), 4096, 33
    row = _randn(g, V, std=2.0)
    ids, _ = _sample(row.expand(n, V).contiguous(), (torch.arange(n) + 0.5) / n, 0.9, 20)
    w = torch.softmax(row.double() / float(torch.tensor(0.9)), 0)
    w[torch.argsort(row, descending=True)[20:]] = 0
    w = w / w.sum()
    share = torch.bincount(ids.long(), minlength=V).double() / n
    assert ((share - w).abs() <= 1.0 / n + 1e-9).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first", [0, 1, 2, 3, 5])
def test_sample_strided_rows(dtype, first):
    """Rows at any distance and alignment."""
    g, n, V = _gen(first), 6, 3001
    wide = torch.full((n, V + 10 + first), 50.0, dtype=dtype, device=DEV)   # what stands beside a row would win
    logits = _logits(g, n, V, dtype)
    wide[:, first:first + V] = logits.to(DEV)
    _check_sample(wide[:, first:first + V], torch.rand(n, generator=g), 1.0, 100, 0.9)
    _check_sample(wide[:, first:first + V], torch.rand(n, generator=g), 1.0, 0, 0.99)


def test_sample_extreme_spreads():
    """Logits whose distance passes every fp32 exponent, and all within a rounding of one another."""
    g, n, V = _gen(9), 6, 4000
    wide = (_randn(g, n, V) * torch.exp(20 * _randn(g, n, V)))
    _check_sample(wide, torch.rand(n, generator=g), 1.0, 50, 0.9)
    _check_sample(wide, torch.rand(n, generator=g), 1e-20)
    close = 1.0 + 2.0 ** -23 * torch.randint(0, 4, (n, V), generator=g)
    _check_sample(close, torch.rand(n, generator=g), 1.0, 1500, 0.7)
    _check_sample(close, torch.rand(n, generator=g), 1e-7, 1500, 0.7)
    _check_sample(torch.randn(n, V, generator=g).abs().neg() * 1e38, torch.rand(n, generator=g), 1e38, 0, 0.9)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_of_the_largest_vocabulary(dtype):
    g, V = _gen(33), 1 << 20
    settings = [(1.0, 0, 1.0, 0.0), (1.0, 64, 0.95, 0.0), (0.7, 0, 0.9, 0.0), (1.5, 0, 0.99, 0.0), (1.0, 50000, 1.0, 0.0),
                (1.0, 0, 1.0, 0.001)]
    t, k, p, m = (list(v) for v in zip(*settings))
    logits = _logits(g, len(settings), V, dtype)
    _check_sample(logits, torch.rand(len(settings), generator=g), t, k, p, m)
    wide = torch.empty(len(settings), V + 3, dtype=dtype, device=DEV)[:, 3:]   # an odd start, and one slice more
    wide.copy_(logits)
    _check_sample(wide, torch.rand(len(settings), generator=g), t, k, p, m)


@pytest.mark.parametrize("n,V", [(100, 100003), (700, 12289), (2100, 4090)])
def test_sample_of_many_slices(n, V):
    """More than 2048 slices of 4096, which are then twice as long."""
    g = _gen(n)
    logits = _logits(g, n, V, F32)
    few = [logits[i] for i in (0, n // 2, n - 1)]
    u = torch.rand(n, generator=g)
    for s in ((1.0, 0, 1.0, 0.0), (0.9, 40, 0.9, 0.0), (1.0, 0, 0.97, 0.0)):
        ids, lp = _sample(logits, u, *s)
        for i, row in zip((0, n // 2, n - 1), few):
            token, want, margin = R.sample_row(row.numpy(), *s, u[i].item())
            assert margin > 2.0 ** -36 and ids[i] == token and abs(lp[i].item() - want) <= 2.0 ** -24 * abs(want) + 1e-8
        one, _ = _sample(logits[n - 1:], u[n - 1:], *s)      # as a call of its own
        assert one[0] == ids[n - 1]


@pytest.mark.parametrize("std", [1e-3, 0.05, 0.4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_crowded_logits(std, dtype):
    """Far more entries within an eighth of a logit than are listed at a time, most of them different (in fp32)."""
    g, V = _gen(17), 90001
    settings = [(1.0, 0, 0.5, 0.0), (1.0, 30000, 0.7, 0.0), (1.0, 30000, 1.0, 0.0), (1.0, 0, 1.0, 0.9), (2.0, 20000, 0.9, 0.5),
                (1.0, 5, 0.5, 0.0), (0.5, 0, 0.9, 0.01), (math.inf, 60000, 0.5, 0.0), (1.0, 2100, 0.9999, 0.0)]
    t, k, p, m = (list(v) for v in zip(*settings))
    logits = _randn(g, len(settings), V, std=std).to(dtype)
    logits[:, ::11] = -math.inf
    for i in range(2):
        _check_sample(logits, torch.rand(len(settings), generator=g), t, k, p, m)


@pytest.mark.parametrize("V", [40, 5000, 60000])
def test_sample_infinite_logits_among_settings(V):
    """Rows with one and several +inf under every rule and temperature: beside them nothing is chosen."""
    g = _gen(V)
    n = len(SETTINGS)
    t, k, p, m = (list(v) for v in zip(*SETTINGS))
    logits = _logits(g, n, V, F32)
    logits[:, V // 3] = math.inf
    logits[::2, V // 2:V // 2 + 9] = math.inf
    logits[:, 0] = torch.finfo(F32).max
    _check_sample(logits, torch.rand(n, generator=g), t, k, p, m)


@pytest.mark.parametrize("T", [1e-45, 1e-40, 1e-37, 1e30, 3e38])
@pytest.mark.parametrize("V", [300, 20011, 60000])
def test_sample_extreme_temperatures(T, V):
    """Temperatures whose inverse passes fp32, and such that all weights are equal; logits of both signs and zeros."""
    g = _gen(V)
    settings = [(0, 1.0, 0.0), (9, 1.0, 0.0), (0, 0.9, 0.0), (40, 0.9, 0.0), (0, 1.0, 0.5), (V - 20, 0.5, 0.1)]
    k, p, m = (list(v) for v in zip(*settings))
    logits = _logits(g, len(settings), V, BF16).float()
    logits[:, 5] = 0.0
    logits[1::2] = -logits[1::2].abs()
    logits[:, ::37] = -math.inf
    _check_sample(logits, torch.rand(len(settings), generator=g), T, k, p, m)


# ------------------------------------------------------------------ positions past 2^31
def test_sample_rows_past_32_bits():
    n, V, stride = 5, 20011, 1 << 30
    g = _gen(3)
    whole = torch.empty(stride * (n - 1) + V, device=DEV)
    logits = whole.as_strided((n, V), (stride, 1))
    logits.copy_(_logits(g, n, V, F32))
    _check_sample(logits, torch.rand(n, generator=g), 1.0, 30, 0.9)
    _check_sample(logits, torch.rand(n, generator=g), 1.0, 0, 0.999)


def test_norm_rows_past_32_bits():
    g, n, dim, stride = _gen(4), 5, 136, 1 << 29
    x = _randn(g, n, dim).bfloat16()
    whole = torch.empty(stride * (n - 1) + dim, dtype=BF16, device=DEV)
    xv = whole.as_strided((n, dim), (stride, 1))
    xv.copy_(x)
    spec = _spec(g, "rms", dim, BF16)
    y = torch.empty(n, dim, dtype=BF16, device=DEV)
    oes.norm(xv, y, pre=spec[0])
    want = R.normed(x.double(), torch.zeros(n, dim, dtype=torch.float64), spec[1])
    _within(y, want[0], R.stored(*want, BF16), "x")
    oes.norm(xv, xv, pre=spec[0])                      # in place, and rows of y as far apart
    assert torch.equal(xv, y)


def test_product_outputs_past_32_bits():
    """n * N above 2^31: the last rows, and some between, against float64."""
    g, n, N, K = _gen(6), 35000, 65537, 16
    x, w = _randn(g, n, K).bfloat16(), _randn(g, N, K).bfloat16()
    y = torch.empty(n, N, dtype=BF16, device=DEV)
    oes.linear_bf16(x.to(DEV), w.to(DEV), y)
    some = torch.tensor([0, 1, n // 2, n - 2, n - 1])
    want, err = R.product(x[some], w, None, "none", 1.0, None)
    _within(y[some.to(DEV)], want, R.stored(want, err, BF16), "rows")


# ------------------------------------------------------------------ graphs, streams, repeats
def _case(seed):
    g = _gen(seed)
    n, D, V = 9, 512, 6001
    s = {"x": _randn(g, n, D).bfloat16().to(DEV), "res": _randn(g, n, D).to(DEV), "w": _randn(g, V, D, std=0.1).bfloat16().to(DEV),
         "wt": (1 + _randn(g, D, std=0.1)).bfloat16().to(DEV), "u": torch.rand(n, generator=g).to(DEV)}
    s["res_out"], s["y"] = torch.empty_like(s["res"]), torch.empty_like(s["x"])
    s["logits"] = torch.empty(n, V, device=DEV)
    s["ids"], s["lp"] = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, device=DEV)
    s["ws"] = torch.empty(oes.sample_workspace_bytes(n, V), dtype=torch.uint8, device=DEV)
    s["k"] = torch.full((n,), 40, dtype=torch.int32, device=DEV)
    s["p"] = torch.full((n,), 0.9, device=DEV)
    s["norm"] = oes.Norm(s["wt"])
    return s


def _pass(s, stream=None):
    oes.norm(s["x"], s["y"], pre=s["norm"], res=s["res"], res_out=s["res_out"], stream=stream)
    oes.linear_bf16(s["y"], s["w"], s["logits"], stream=stream)
    oes.sample(s["logits"], s["u"], s["ids"], s["ws"], top_k=s["k"], top_p=s["p"], logprob=s["lp"], stream=stream)


OUT = ("res_out", "y", "logits", "ids", "lp")


def test_repeats_and_other_streams_agree():
    s = _case(1)
    _pass(s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUT}
    for i in range(3):
        for k in OUT:
            s[k].fill_(3)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if i == 0:
            _pass(s, stream=side)
        else:
            with torch.cuda.stream(side):
                _pass(s)
        torch.cuda.current_stream().wait_stream(side)
        for k in OUT:
            assert torch.equal(s[k], want[k]), (i, k)


def test_captured_steps_replay():
    """Two graphs with a workspace each, replayed on new inputs between eager calls."""
    a, b = _case(2), _case(3)
    for s in (a, b):
        _pass(s)
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _pass(s)
        graphs.append(graph)
    for i in range(4):
        fresh = [_case(10 + 2 * i), _case(11 + 2 * i)]
        for s, f in zip((a, b), fresh):
            for k in ("x", "res", "w", "wt", "u"):
                s[k].copy_(f[k])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for s, f in zip((a, b), fresh):
            _pass(f)
            for k in OUT:
                assert torch.equal(s[k], f[k]), (i, k)


def test_no_rows():
    e = torch.empty
    oes.norm(e(0, 64, dtype=BF16, device=DEV), e(0, 64, dtype=BF16, device=DEV), pre=oes.Norm())
    oes.linear_bf16(e(0, 64, dtype=BF16, device=DEV), e(5, 64, dtype=BF16, device=DEV), e(0, 5, dtype=BF16, device=DEV))
    oes.sample(e(0, 5, device=DEV), e(0, device=DEV), e(0, dtype=torch.int32, device=DEV), e(16, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ a decode step of all of them
def _held(got, y, err, kind, what):
    _within(got, y, R.stored(y, err, kind), what)


@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_from_hidden_state_to_token(captured):
    """Steps of a small model whose layer is made of these operators and those around the expert step: every
    output of every step against float64 on that step's own inputs; the sampled token is the next one's input."""
    g = _gen(21)
    B, H, heads, kvh, D, I, V, L = 3, 256, 8, 2, 32, 192, 1003, 2
    page, steps = 16, 4
    embed = _randn(g, V, H).bfloat16().to(DEV)
    qkv_n = (heads + 2 * kvh) * D

    def weights(*shape):
        return _randn(g, *shape, std=1.0 / math.sqrt(shape[-1])).bfloat16().to(DEV)

    layers = []
    for _ in range(L):
        layers.append({"n1": _spec(g, "rms", H, BF16), "n2": _spec(g, "rms", H, BF16), "post": _spec(g, "rms", H, BF16),
                       "qn": _spec(g, "rms", D, BF16), "qkv": weights(qkv_n, H), "bias": weights(1, qkv_n)[0],
                       "o": weights(H, heads * D), "gu": weights(2 * I, H), "down": weights(H, I), "sg": weights(1, H),
                       "k": torch.zeros(2 * B, page, kvh, D, dtype=BF16, device=DEV),
                       "v": torch.zeros(2 * B, page, kvh, D, dtype=BF16, device=DEV)})
    final = _spec(g, "rms", H, BF16)
    head = weights(V, H)
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    length = torch.zeros(B, dtype=torch.int32, device=DEV)
    q_start = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    freq = torch.tensor(oes.rope_freqs(D)[0], device=DEV)
    for l in layers:
        l["kv"] = oes.KvPages(l["k"], l["v"], table, length)
    need = max(oes.attn_workspace_bytes(layers[0]["kv"], heads, B), 16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    sws = torch.empty(oes.sample_workspace_bytes(B, V), dtype=torch.uint8, device=DEV)
    ids, lp, u = torch.zeros(B, dtype=torch.int32, device=DEV), torch.empty(B, device=DEV), torch.empty(B, device=DEV)
    top_k, top_p = torch.full((B,), 40, dtype=torch.int32, device=DEV), torch.full((B,), 0.95, device=DEV)
    log = []

    def bf(*shape):
        return torch.empty(*shape, dtype=BF16, device=DEV)

    def step():
        log.clear()
        x, res = embed[ids.long()], None
        for l in layers:
            y, stream_ = bf(B, H), torch.empty(B, H, device=DEV)
            if res is None:
                oes.norm(x, y, pre=l["n1"][0], res_out=stream_)
                log.append(("norm", x, l["n1"][1], None, None, 1.0, None, stream_, y))
            else:
                gate = bf(B, 1)
                oes.linear_bf16(x, l["sg"], gate, act="sigmoid")
                log.append(("product", x, l["sg"], None, "sigmoid", 1.0, None, gate))
                oes.norm(x, y, pre=l["n1"][0], post=l["post"][0], gate=gate, scale=0.5, res=res, res_out=stream_)
                log.append(("norm", x, l["n1"][1], l["post"][1], gate, 0.5, res, stream_, y))
            qkv = bf(B, qkv_n)
            oes.linear_bf16(y, l["qkv"], qkv, bias=l["bias"])
            log.append(("product", y, l["qkv"], l["bias"], "none", 1.0, None, qkv))
            parts = qkv.view(B, heads + 2 * kvh, D)
            q, k, v = parts[:, :heads], parts[:, heads:heads + kvh], parts[:, heads + kvh:]
            qn = bf(B, heads, D)
            oes.norm(q, qn, pre=l["qn"][0])
            log.append(("norm", q, l["qn"][1], None, None, 1.0, None, None, qn))
            oes.rope_append(qn, qn2 := bf(B, heads, D), k, v, freq, pos, l["kv"], q_start)
            out = bf(B, heads, D)
            oes.attn(qn2, out, l["kv"], q_start, 1 / math.sqrt(D), ws)
            o, flat = bf(B, H), out.view(B, heads * D)
            oes.linear_bf16(flat, l["o"], o, scale=0.7)
            log.append(("product", flat, l["o"], None, "none", 0.7, None, o))
            y2, r2 = bf(B, H), torch.empty(B, H, device=DEV)
            oes.norm(o, y2, pre=l["n2"][0], res=stream_, res_out=r2)
            log.append(("norm", o, l["n2"][1], None, None, 1.0, stream_, r2, y2))
            h = bf(B, I)
            oes.linear_bf16(y2, l["gu"], h, act="swiglu")
            log.append(("product", y2, l["gu"], None, "swiglu", 1.0, None, h))
            x, res = bf(B, H), r2
            oes.linear_bf16(h, l["down"], x)
            log.append(("product", h, l["down"], None, "none", 1.0, None, x))
        y = bf(B, H)
        oes.norm(x, y, pre=final[0], res=res)
        log.append(("norm", x, final[1], None, None, 1.0, res, None, y))
        logits = torch.empty(B, V, device=DEV)
        oes.linear_bf16(y, head, logits, scale=2.0)
        log.append(("product", y, head, None, "none", 2.0, None, logits))
        oes.sample(logits, u, ids, sws, top_k=top_k, top_p=top_p, logprob=lp)
        log.append(("sample", logits))

    def clear():
        for l in layers:
            l["k"].zero_()
            l["v"].zero_()

    if captured:
        length.fill_(1)
        u.fill_(0.5)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        clear()
    ids.copy_(torch.tensor([1, 500, V - 1], dtype=torch.int32))
    tokens = []
    for i in range(steps):
        length.fill_(i + 1)
        pos.fill_(i)
        u.copy_(torch.rand(B, generator=g))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        for at, (op, x, *rest) in enumerate(log):
            what = (i, at, op)
            if op == "norm":
                pre, post, gate, scale, res, stream_, y = rest
                r, err = R.norm(x, post, gate, "plain", scale, res)
                if stream_ is not None:
                    _held(stream_, r, err, F32, what)
                    r, err = stream_.double().cpu(), torch.zeros_like(r)
                _held(y, *R.normed(r, err, pre), BF16, what)
            elif op == "product":
                w, bias, act, scale, res, y = rest
                _held(y, *R.product(x, w, bias, act, scale, res), y.dtype, what)
            else:
                rows, us = x.cpu().numpy(), u.cpu()
                for b in range(B):
                    token, want, margin = R.sample_row(rows[b], 1.0, 40, float(top_p[b]), 0.0, us[b].item())
                    assert margin > 2.0 ** -36 and ids[b] == token and abs(lp[b].item() - want) < 1e-6, (what, b)
        for l in layers:
            l["kv"].check()
        tokens.append(ids.tolist())
    assert len(set(map(tuple, tokens))) > 1

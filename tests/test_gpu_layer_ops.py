"""The operators around the expert step on the GPU, against float64 references: every type,
layout and mask at small sizes, empty rows, ragged and odd shapes, strides, garbage in
places that no row sees, bad pages, repeats and graphs."""
import math

import numpy as np
import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _starts(q):
    return [0] + list(np.cumsum(q))


def _dev32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _within(got, ref, bound, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


# ------------------------------------------------------------------ linear
def _banks(fmt, N, K, seed):
    g = _gen(seed)
    if fmt == "mxfp4_t":
        return [torch.randint(0, 256, (K // 32, N, 16), dtype=torch.uint8, generator=g),
                torch.randint(110, 125, (K // 32, N), dtype=torch.uint8, generator=g), torch.randn(N, generator=g).bfloat16()]
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    if fmt == "q4_0":
        return [codes, (0.01 * torch.randn(N, K // 32, generator=g)).half()]
    return [codes, torch.randint(0, 0x7f, (N, K // 16), dtype=torch.uint8, generator=g),
            (1e-3 * torch.randn(N, generator=g)).half()]


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4", "mxfp4_t"])
@pytest.mark.parametrize("n,N,K", [(1, 1, 32), (1, 17, 96), (1, 515, 2048), (1, 64, 7168), (2, 33, 160), (3, 1030, 256),
                                   (5, 16, 1024), (8, 100, 2880), (15, 47, 416), (16, 256, 512), (17, 129, 128),
                                   (33, 80, 544), (64, 31, 2048), (65, 200, 192), (200, 48, 64)])
def test_linear(fmt, n, N, K):
    banks = _banks(fmt, N, K, n * N + K)
    x = torch.randn(n, K, generator=_gen(K)).bfloat16()
    wide = torch.full((n, N + 3), 7.0, dtype=torch.bfloat16, device=DEV)
    xs = torch.zeros(n, K + 8, dtype=torch.bfloat16, device=DEV)
    xs[:, :K] = x.to(DEV)
    oes.linear(fmt, xs[:, :K], [b.to(DEV) for b in banks], wide[:, :N])
    ref, bound = R.linear(fmt, x, banks, N)
    _within(wide[:, :N], ref, bound, (fmt, n, N, K))
    assert (wide[:, N:] == 7).all(), "written behind the row"


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4", "mxfp4_t"])
@pytest.mark.parametrize("n,N,K", [(23, 5529, 288), (1, 5003, 4128), (3, 9999, 2912), (2, 20005, 2080), (9, 24600, 288),
                                   (16, 24577, 1536), (20, 24600, 800), (40, 24593, 800), (70, 24611, 256)])
def test_linear_many_rows(fmt, n, N, K):
    """Waves of rows past the last one, with a short last step of K; every split of the waves, x in pieces."""
    banks = _banks(fmt, N, K, n + K)
    x = torch.randn(n, K, generator=_gen(K)).bfloat16()
    y = torch.full((n + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    oes.linear(fmt, x.to(DEV), [b.to(DEV) for b in banks], y[:n])
    ref, bound = R.linear(fmt, x, banks, N)
    _within(y[:n], ref, bound, (fmt, n, N, K))
    assert (y[n] == 7).all()


@pytest.mark.parametrize("n", [1, 4, 9])
def test_linear_extremes(n):
    """Large activations in one block, zero blocks, NaN and infinite scales reach their rows only."""
    N, K = 40, 256
    for fmt in ("q4_0", "nvfp4", "mxfp4_t"):
        banks = _banks(fmt, N, K, 5)
        x = torch.randn(n, K, generator=_gen(6)).bfloat16()
        x[:, 37] = 3e4
        x[0, :32] = 0
        if fmt == "mxfp4_t":
            banks[1][1, 3], banks[1][2, 5], banks[1][0, 6] = 255, 0, 1
            banks[2] = None
        elif fmt == "nvfp4":
            banks[1][3, 2] = 0x7f
        else:
            banks[1][3, 2] = math.inf
        y = torch.empty(n, N, dtype=torch.bfloat16, device=DEV)
        oes.linear(fmt, x.to(DEV), [b if b is None else b.to(DEV) for b in banks], y)
        ref, bound = R.linear(fmt, x, banks, N)
        fine = torch.arange(N) != 3
        assert not y[:, 3].isfinite().any()
        _within(y[:, fine.to(DEV)], ref[:, fine], bound[:, fine], fmt)


# ------------------------------------------------------------------ rope
ROPE = [("half", "none", 64, 64), ("interleaved", "none", 64, 64), ("half", "linear", 128, 128), ("interleaved", "yarn", 128, 64),
        ("half", "ntk", 128, 96), ("half", "none", 80, 26), ("interleaved", "linear", 96, 42), ("half", "yarn", 256, 2),
        ("interleaved", "none", 16, 16), ("half", "none", 112, 36), ("half", "none", 64, 32)]


def _rope_bound(x, ref):
    """Half a bf16 step, and fp32: sine and cosine off by 2^-22 (4 U, of values up to mscale), two products and a sum."""
    mag = x.double().abs().amax(-1, keepdim=True) * 2 * 1.5
    return R.BF * ref.abs() + (1 + R.BF) * 8 * R.U * mag


@pytest.mark.parametrize("layout,scaling,D,rot", ROPE)
@pytest.mark.parametrize("n,heads,in_place", [(1, 1, False), (7, 5, True), (65, 3, False)])
def test_rope(layout, scaling, D, rot, n, heads, in_place):
    g = _gen(D + rot + n)
    freq, m = oes.rope_freqs(rot, 10000.0, scaling, 8.0, 2048)
    freq = torch.from_numpy(freq)
    fused = torch.randn(n, heads + 2, D, generator=g).bfloat16()
    x = fused[:, 1:heads + 1]
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g).int()
    pos[0] = 0
    if n > 3:
        pos[1], pos[2], pos[3] = 2 ** 31 - 1, 1, -5
    dx = fused.to(DEV)
    y = dx[:, 1:heads + 1] if in_place else torch.full((n, heads, D), 9.0, dtype=torch.bfloat16, device=DEV)
    oes.rope(dx[:, 1:heads + 1], y, freq.to(DEV), pos.to(DEV), layout, m)
    ref = R.turn(x, pos, freq, m, layout, rot)
    _within(y, ref, _rope_bound(x, ref), (layout, scaling, D, rot))
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:]), "values behind rot_dim are copied"
    keep = [0, heads + 1] if in_place else range(heads + 2)
    assert all(torch.equal(dx[:, i].cpu(), fused[:, i]) for i in keep), "neighbours changed"


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout,D,rot,page,head_major", [("half", 64, 64, 16, False), ("interleaved", 128, 64, 7, True),
                                                          ("half", 80, 26, 1, False), ("interleaved", 96, 96, 64, True)])
def test_rope_append(elem, layout, D, rot, page, head_major):
    """Tokens of ragged sequences into their entries; a sequence without tokens, one whose first
    tokens have no entry, spare rows; everything else in the cache stays."""
    q_len, lens = [3, 0, 40, 5, 1], [9, 4, 40, 2, 33]
    Hq, Hkv, spare, g = 6, 2, 2, _gen(D)
    c = R.Cache(1, lens, Hkv, D, page, elem, head_major)
    start = _starts(q_len)
    n = start[-1]
    q = torch.randn(n + spare, Hq, D, generator=g).bfloat16()
    k, v = torch.randn(n, Hkv, D, generator=g).bfloat16(), torch.randn(n, Hkv, D, generator=g).bfloat16()
    v[0, 0, 0], v[1, 0, 1], k[2, 1, D - 1] = 1e4, math.nan, -1e4
    freq, m = oes.rope_freqs(rot, 10000.0, "yarn", 4.0, 1024)
    freq = torch.from_numpy(freq)
    pos = torch.randint(0, 1 << 20, (n,), generator=g).int()
    kv = c.handle(oes)
    q_out = torch.full((n + spare, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    oes.rope_append(q.to(DEV), q_out, k.to(DEV), v.to(DEV), freq.to(DEV), pos.to(DEV), kv, _dev32(start), layout, m)
    kv.check()
    ref_q = R.turn(q[:n], pos, freq, m, layout, rot)
    _within(q_out[:n], ref_q, _rope_bound(q[:n], ref_q), "q")
    assert (q_out[n:] == 9).all()
    new_k, new_v = R.turn(k, pos, freq, m, layout, rot), v.double()
    bound = _rope_bound(k, new_k)
    got_k, got_v = c.dk.cpu().float().double(), c.dv.cpu().float().double()
    old_k, old_v = c.k.float().double(), c.v.float().double()
    for b, (a, e) in enumerate(zip(q_len, lens)):
        for i in range(a):
            j, t = e - a + i, start[b] + i
            if j < 0:
                continue
            p, r = int(c.table[b, j // page]), j % page
            if elem == "bf16":
                _within(got_k[p, r], new_k[t], bound[t], "k")
                assert torch.equal(got_v[p, r].nan_to_num(5), new_v[t].nan_to_num(5))
            else:
                want = R.to_e4m3((v[t].float() / torch.tensor(c.v_scale)).double())
                assert torch.equal(got_v[p, r].nan_to_num(5), want.nan_to_num(5))
                # the rotated fp32 value may fall on the other side of a rounding border
                lo, hi = ((new_k[t] - bound[t] - 1e-9) / c.k_scale).clamp(-448, 448), ((new_k[t] + bound[t] + 1e-9) / c.k_scale).clamp(-448, 448)
                assert ((got_k[p, r] >= R.to_e4m3(lo)) & (got_k[p, r] <= R.to_e4m3(hi))).all()
            old_k[p, r], old_v[p, r] = got_k[p, r], got_v[p, r]
    assert torch.equal(old_k.nan_to_num(5), got_k.nan_to_num(5)) and torch.equal(old_v.nan_to_num(5), got_v.nan_to_num(5)), "another entry changed"


# ------------------------------------------------------------------ attn and weigh
CASES = [
    # heads, kv_heads, D, page, elem, window, q_len, lens
    (4, 1, 64, 16, "bf16", 0, [1], [1]),
    (8, 2, 128, 16, "bf16", 0, [1, 1, 1], [33, 1, 700]),
    (32, 4, 128, 64, "e4m3", 0, [1, 1], [1029, 64]),
    (16, 2, 64, 1, "bf16", 0, [3, 1, 0, 2], [65, 2, 9, 2]),
    (5, 5, 48, 7, "bf16", 0, [2, 9], [130, 9]),
    (6, 2, 80, 16, "e4m3", 0, [17, 1], [40, 300]),
    (8, 8, 96, 32, "bf16", 5, [70, 3], [100, 3]),
    (12, 2, 112, 100, "bf16", 64, [33, 128, 1], [333, 128, 500]),
    (8, 1, 256, 16, "bf16", 0, [40, 1], [200, 77]),
    (2, 1, 192, 16, "e4m3", 33, [65], [190]),
    (128, 1, 64, 16, "bf16", 0, [3, 1], [70, 200]),
    (40, 1, 16, 16, "bf16", 0, [5], [300]),
    (3, 1, 32, 64, "e4m3", 1, [9, 4], [9, 64]),
    (8, 2, 128, 16, "bf16", 0, [200, 0, 7], [459, 12, 600]),
    (64, 8, 64, 32, "bf16", 128, [130, 1], [1000, 131]),
    (16, 4, 128, 64, "e4m3", 0, [150], [2300]),
    (8, 2, 64, 16, "bf16", 0, [6, 3], [2, 0]),      # rows before entry 0: they see nothing
    (4, 4, 128, 16, "bf16", 0, [1, 1], [5000, 4097]),
]


def _attn_case(case, seed=0, head_major=False, fill=math.nan, spare=3):
    Hq, Hkv, D, page, elem, window, q_len, lens = case
    c = R.Cache(seed, lens, Hkv, D, page, elem, head_major, fill=fill)
    start = _starts(q_len)
    q = torch.randn(start[-1] + spare, Hq, D, generator=_gen(seed + 1)).bfloat16()
    return c, start, q, 1.0 / math.sqrt(D), window


def _run_attn(c, start, q, scale, window, kv=None, stream=None):
    kv = kv or c.handle(oes)
    n, Hq, D = q.shape
    fused = torch.full((n, Hq + 1, D), 5.0, dtype=torch.bfloat16, device=DEV)
    dq = torch.zeros(n, Hq + 3, D, dtype=torch.bfloat16, device=DEV)
    dq[:, 2:Hq + 2] = q.to(DEV)
    out, lse = fused[:, :Hq], torch.full((n, Hq), 5.0, device=DEV)
    ws = torch.full((oes.attn_workspace_bytes(kv, Hq, n) + 64,), 255, dtype=torch.uint8, device=DEV)  # NaN bytes
    oes.attn(dq[:, 2:Hq + 2], out, kv, _dev32(start), scale, ws, window, lse)
    assert (fused[:, Hq] == 5).all(), "written beside the output"
    assert (ws[-64:] == 255).all(), "written behind the workspace"
    return kv, dq[:, 2:Hq + 2], out, lse


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attn(case, head_major):
    c, start, q, scale, window = _attn_case(case, 3, head_major)
    kv, _, out, lse = _run_attn(c, start, q, scale, window)
    n = start[-1]
    ref, ref_lse, bound, _ = R.attention(q, c, start, scale, window)
    _within(out[:n], ref[:n], bound[:n], case)
    assert (out[n:] == 5).all() and (lse[n:] == 5).all(), "rows behind the last sequence"
    got = lse[:n].double().cpu()
    empty = ref_lse[:n] == -math.inf
    assert torch.equal(got == -math.inf, empty)
    assert (out[:n].cpu()[empty] == 0).all()
    # a score is off by (D + 4) U sum |q k| scale <= (D + 4) U * 8 sqrt(D) here, the log by 8 U of its value
    lim = (q.shape[2] + 4) * R.U * 8 * math.sqrt(q.shape[2]) + 8 * R.U * (1 + ref_lse[:n].abs())
    assert ((got - ref_lse[:n]).abs() <= lim)[~empty].all()
    kv.check()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attn_weigh(case):
    c, start, q, scale, window = _attn_case(case, 5)
    kv = c.handle(oes)
    Hq, Hkv, D = case[0], case[1], case[2]
    n = start[-1]
    _, ref_lse, _, p = R.attention(q, c, start, scale, window)
    lse = torch.full(q.shape[:2], math.nan)
    lse[:n] = ref_lse[:n].float()
    cap = c.cols * c.page + 5
    acc = torch.rand(len(c.lens), Hkv, cap, generator=_gen(8))
    dacc = acc.to(DEV)
    oes.attn_weigh(q.to(DEV), lse.to(DEV), kv, _dev32(start), scale, dacc, window)
    got = dacc.cpu()
    for b, m in enumerate(c.lens):
        add = p[b].view(p[b].shape[0], Hkv, Hq // Hkv, m).sum((0, 2))
        rows = max(1, p[b].shape[0] * (Hq // Hkv))
        ref = acc[b, :, :m].double() + add
        # a weight is off by twice its score's error (see test_attn) and the lse's rounding; sums of `rows` terms
        rel = 2 * ((D + 4) * R.U * 8 * math.sqrt(D) + 16 * R.U) + (rows + 2) * R.U
        _within(got[b, :, :m], ref, rel * add + 2 * R.U * ref + 1e-30, (case, b))
        assert torch.equal(got[b, :, m:], acc[b, :, m:]), "written behind the sequence"
    kv.check()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,window,q_len,lens", [(8, 2, 64, 0, [6, 1], [80, 33]), (4, 4, 128, 40, [150], [300]),
                                                      (64, 1, 64, 0, [5], [70]), (8, 1, 128, 0, [130], [130])])
def test_what_a_row_does_not_see_does_not_reach_it(bad, elem, Hq, Hkv, D, window, q_len, lens):
    """A key and a value that are NaN or infinite at the last entry reach the last row alone (and with a
    window, those at entry 0 no row behind it): every other row is as without them."""
    if elem == "e4m3" and bad != bad or elem == "bf16":
        c, start, q, scale, _ = _attn_case((Hq, Hkv, D, 16, elem, window, q_len, lens), 7)
        _, _, clean, lse0 = _run_attn(c, start, q, scale, window)
        clean, lse0 = clean.clone(), lse0.clone()
        for b, m in enumerate(lens):
            for j in [m - 1] + ([0] if window and m - q_len[b] - window > 0 else []):
                p, r = int(c.table[b, j // 16]), j % 16
                if elem == "bf16":
                    c.dk[p, r], c.dv[p, r] = bad, bad
                else:
                    c.dk.view(torch.uint8)[p, r], c.dv.view(torch.uint8)[p, r] = 0x7f, 0x7f
        _, _, out, lse = _run_attn(c, start, q, scale, window)
        last = torch.zeros(q.shape[0], dtype=torch.bool)
        for b in range(len(lens)):
            last[start[b + 1] - 1] = True
        n = start[-1]
        rest = (~last[:n]).nonzero()[:, 0].to(DEV)
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], lse0[rest])
        if bad != bad:
            assert out[last.nonzero()[:, 0].to(DEV)].isnan().all()


def test_values_that_rows_see_are_not_hidden():
    """An infinite value at an entry that all later rows see: infinite (of its sign) there, finite before."""
    c, start, q, scale, _ = _attn_case((4, 2, 64, 16, "bf16", 0, [100], [100]), 9)
    p, r = int(c.table[0, 40 // 16]), 40 % 16
    c.dv[p, r, :, 3] = -math.inf
    _, _, out, _ = _run_attn(c, start, q, scale, 0)
    assert out[:40].isfinite().all() and out[40:100, :, :3].isfinite().all() and out[40:100, :, 4:].isfinite().all()
    assert (out[40:100, :, 3] == -math.inf).all()


@pytest.mark.parametrize("scale", [1e-6, 3.0, 60.0])
def test_attn_score_ranges(scale):
    """Flat and very sharp softmaxes (scores of several thousand)."""
    c, start, q, _, _ = _attn_case((8, 2, 128, 16, "bf16", 0, [33, 1], [300, 500]), 11)
    _, _, out, lse = _run_attn(c, start, q, scale, 0)
    n = start[-1]
    ref, ref_lse, bound, _ = R.attention(q, c, start, scale)
    _within(out[:n], ref[:n], bound[:n], scale)
    assert torch.allclose(lse[:n].double().cpu(), ref_lse[:n], rtol=1e-5, atol=1e-5)


def test_bad_pages_lengths_and_rows():
    """Entries of bad pages count as masked in attn and weigh, are not written by rope_append, and keep a
    sequence out of an eviction; lengths and row ranges are clamped; each raises the status."""
    case = (8, 2, 64, 16, "bf16", 0, [1, 40], [100, 90])
    c, start, q, scale, _ = _attn_case(case, 13)
    c.table[0, 2], c.table[1, 0], c.table[1, 5] = c.pages, -7, 2 ** 31 - 1
    c.to(DEV)
    kv, dq, out, lse = _run_attn(c, start, q, scale, 0)
    with pytest.raises(oes.OesError) as e:
        kv.check()
    assert e.value.status == oes.ERR_ARG
    kv.check()  # cleared
    n = start[-1]
    ref, ref_lse, bound, p = R.attention(q, c, start, scale)
    _within(out[:n], ref[:n], bound[:n], "pages")
    acc = torch.zeros(2, 2, c.cols * 16, device=DEV)
    lse32 = torch.zeros(q.shape[:2])
    lse32[:n] = ref_lse[:n].float()
    oes.attn_weigh(dq.contiguous(), lse32.to(DEV), kv, _dev32(start), scale, acc)
    add = p[1].view(-1, 2, 4, 90).sum((0, 2))
    assert torch.allclose(acc[1, :, :90].double().cpu(), add, rtol=1e-4, atol=1e-6)
    with pytest.raises(oes.OesError):
        kv.check()
    k0, v0 = c.dk.clone(), c.dv.clone()
    kept, new_len = torch.empty(2, 2, 50, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(oes.kv_evict_workspace_bytes(kv, 50), dtype=torch.uint8, device=DEV)
    oes.kv_evict(kv, acc, 50, kept, new_len, ws)
    assert (kept == -1).all() and new_len.tolist() == [100, 90]
    assert torch.equal(c.dk.nan_to_num(5), k0.nan_to_num(5)) and torch.equal(c.dv.nan_to_num(5), v0.nan_to_num(5))
    with pytest.raises(oes.OesError):
        kv.check()
    freq = torch.from_numpy(oes.rope_freqs(64)[0]).to(DEV)
    k = torch.ones(n, 2, 64, dtype=torch.bfloat16, device=DEV)
    c.table[1, 4] = -1
    c.dtable.copy_(c.table)
    oes.rope_append(dq[:n].contiguous(), out[:n].contiguous(), k, k, freq, torch.zeros(n, dtype=torch.int32, device=DEV), kv, _dev32(start))
    with pytest.raises(oes.OesError):
        kv.check()
    touched = (c.dv == 1).all(-1).all(-1).nonzero().tolist()
    assert sorted(touched) == sorted([[int(c.table[b, j // 16]), j % 16] for b, a, m in ((0, 1, 100), (1, 40, 90))
                                      for j in range(m - a, m) if 0 <= c.table[b, j // 16] < c.pages])

    # lengths beyond the table and below zero, row ranges that run backwards or past the rows
    c = R.Cache(2, [64, 48], 2, 64, 16)
    c.dlen.copy_(_dev32([70, -3]))
    kv = c.handle(oes)
    q = torch.randn(6, 4, 64, generator=_gen(1)).bfloat16()
    _run_attn(c, [0, 2, 4], q, 0.125, 0, kv)
    with pytest.raises(oes.OesError):
        kv.check()
    for start in ([0, 5, 3], [-2, 1, 2], [0, 2, 9]):
        c.dlen.copy_(_dev32([64, 48]))
        _, _, out, _ = _run_attn(c, start, q, 0.125, 0, kv)
        assert out.isfinite().all()
        with pytest.raises(oes.OesError):
            kv.check()


# ------------------------------------------------------------------ evict
@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D,page,head_major,budget,first,last,lens", [
    (1, 64, 16, False, 1, 0, 0, [2, 1, 0, 7]), (2, 128, 16, True, 20, 4, 8, [21, 20, 100, 3]),
    (3, 80, 7, False, 33, 0, 33, [34, 200]), (2, 256, 64, True, 64, 64, 0, [65, 300]),
    (2, 16, 1, False, 100, 3, 5, [1025, 2049, 101]), (4, 128, 16, False, 700, 2, 100, [5000, 700, 1024]),
    (1, 96, 32, True, 1500, 0, 0, [3000]), (2, 64, 16, False, 5000, 1, 1, [300, 20])])
def test_evict(elem, Hkv, D, page, head_major, budget, first, last, lens):
    c = R.Cache(17, lens, Hkv, D, page, elem, head_major)
    cap = c.cols * page + 2
    g = _gen(4)
    acc = torch.rand(len(lens), Hkv, cap, generator=g)
    acc[:, :, ::3] = (acc[:, :, ::3] * 4).round() / 4     # many equal weights
    acc[0, 0, :8:2], acc[0, 0, 1:8:2] = 0.0, -0.0
    if cap > 40:
        acc[0, 0, 30:34] = torch.tensor([math.nan, math.inf, -1.0, -math.inf])
    kv = c.handle(oes)
    dacc = acc.to(DEV)
    kept = torch.full((len(lens), Hkv, budget), 77, dtype=torch.int32, device=DEV)
    new_len = torch.empty(len(lens), dtype=torch.int32, device=DEV)
    ws = torch.full((oes.kv_evict_workspace_bytes(kv, budget),), 255, dtype=torch.uint8, device=DEV)
    oes.kv_evict(kv, dacc, budget, kept, new_len, ws, first, last)
    kv.check()
    ref = R.evict(acc, lens, c, budget, first, last)
    assert torch.equal(kept.cpu(), ref)
    assert new_len.tolist() == [min(m, budget) for m in lens]
    bits = torch.int16 if elem == "bf16" else torch.uint8
    k, v = c.k.contiguous().view(bits).clone(), c.v.contiguous().view(bits).clone()
    k0, v0, a = k.clone(), v.clone(), acc.clone()
    for b, m in enumerate(lens):
        if m <= budget:
            continue
        to = torch.arange(budget)
        for h in range(Hkv):
            src = ref[b, h].long()
            for x, x0 in ((k, k0), (v, v0)):
                x[c.table[b, to // page].long(), to % page, h] = x0[c.table[b, src // page].long(), src % page, h]
            a[b, h, to] = acc[b, h, src]
    assert torch.equal(c.dk.cpu().contiguous().view(bits), k) and torch.equal(c.dv.cpu().contiguous().view(bits), v)
    assert torch.equal(dacc.cpu().nan_to_num(9.0), a.nan_to_num(9.0))


def test_evict_into_the_length_itself():
    c = R.Cache(19, [90, 10], 2, 64, 16)
    kv = c.handle(oes)
    acc = torch.rand(2, 2, c.cols * 16, device=DEV)
    kept = torch.empty(2, 2, 40, dtype=torch.int32, device=DEV)
    ws = torch.empty(oes.kv_evict_workspace_bytes(kv, 40), dtype=torch.uint8, device=DEV)
    for _ in range(2):
        oes.kv_evict(kv, acc, 40, kept, c.dlen, ws, 1, 4)
        assert c.dlen.tolist() == [40, 10]


# ------------------------------------------------------------------ together
def _layer(seed=0):
    """A small decoder layer's attention half: weights, cache and a decode loop's buffers."""
    H, Hq, Hkv, D, B, page, budget = 256, 8, 2, 64, 3, 16, 48
    g = _gen(seed)
    wq = [b.to(DEV) for b in _banks("q4_0", (Hq + 2 * Hkv) * D, H, 1)]
    wo = [b.to(DEV) for b in _banks("nvfp4", H, Hq * D, 2)]
    c = R.Cache(3, [page * 8] * B, Hkv, D, page)
    c.dlen.copy_(_dev32([5, 40, 47]))
    f, m = oes.rope_freqs(D, 10000.0, "linear", 2.0)
    d = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, budget=budget, wq=wq, wo=wo, c=c, kv=c.handle(oes), freq=torch.from_numpy(f).to(DEV),
             x=torch.randn(B, H, generator=g).bfloat16().to(DEV), pos=_dev32([5, 40, 47]), start=_dev32([0, 1, 2, 3]))
    n = (Hq + 2 * Hkv) * D
    d["qkv"] = torch.empty(B, n, dtype=torch.bfloat16, device=DEV)
    d["out"], d["y"] = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, dtype=torch.bfloat16, device=DEV)
    d["lse"], d["acc"] = torch.empty(B, Hq, device=DEV), torch.zeros(B, Hkv, page * 8, device=DEV)
    d["kept"] = torch.empty(B, Hkv, budget, dtype=torch.int32, device=DEV)
    d["ws"] = torch.empty(max(16, oes.attn_workspace_bytes(d["kv"], Hq, B)), dtype=torch.uint8, device=DEV)
    d["ews"] = torch.empty(oes.kv_evict_workspace_bytes(d["kv"], budget), dtype=torch.uint8, device=DEV)
    return d


def _layer_step(d, stream=None):
    """x -> q, k, v -> rope into the cache -> attention -> weights -> output projection -> eviction."""
    Hq, Hkv, D = d["Hq"], d["Hkv"], d["D"]
    oes.linear("q4_0", d["x"], d["wq"], d["qkv"], stream=stream)
    qkv = d["qkv"].view(d["B"], Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    oes.rope_append(q, q, k, v, d["freq"], d["pos"], d["kv"], d["start"], stream=stream)
    oes.attn(q, d["out"], d["kv"], d["start"], D ** -0.5, d["ws"], lse=d["lse"], stream=stream)
    oes.attn_weigh(q, d["lse"], d["kv"], d["start"], D ** -0.5, d["acc"], stream=stream)
    oes.linear("nvfp4", d["out"].view(d["B"], -1), d["wo"], d["y"], stream=stream)
    oes.kv_evict(d["kv"], d["acc"], d["budget"], d["kept"], d["c"].dlen, d["ews"], 2, 8, stream=stream)


def test_a_decode_loop():
    """Eight steps of the layer: every step's attention and projection against the float64 reference on the
    state that the step found, the cache's growth and its cuts."""
    d = _layer()
    c = d["c"]
    lens = [5, 40, 47]
    for step in range(8):
        lens = [m + 1 for m in lens]
        c.dlen.copy_(_dev32(lens))
        d["acc"][torch.arange(3), :, torch.tensor(lens) - 1] = 0
        c.lens = lens
        _layer_step(d)
        d["kv"].check()
        lens = [min(m, 48) for m in lens]
        assert c.dlen.tolist() == lens
        qkv, bound = R.linear("q4_0", d["x"], d["wq"], d["qkv"].shape[1])
        v = d["qkv"].double().cpu()[:, -2 * 64:]
        assert ((v - qkv[:, -2 * 64:]).abs() <= bound[:, -2 * 64:]).all()
        y, bound = R.linear("nvfp4", d["out"].view(3, -1), d["wo"], d["y"].shape[1])
        _within(d["y"], y, bound, "output projection")
        # every row's weights sum to one in each query head: to the number of heads of a group in all
        d["x"] = (d["y"].float() / (1e-3 + d["y"].float().square().mean(-1, keepdim=True).sqrt())).bfloat16()
        d["pos"] += 1


def test_a_decode_loop_against_plain_attention():
    d = _layer(3)
    c, lens = d["c"], [6, 41, 48]
    c.dlen.copy_(_dev32(lens))
    d["budget"] = 48
    _layer_step(d)
    c.lens, c.k, c.v = lens, c.dk.cpu(), c.dv.cpu()
    q = d["qkv"].view(3, 12, 64)[:, :8].cpu()
    ref, _, bound, p = R.attention(q, c, [0, 1, 2, 3], 64 ** -0.5)
    _within(d["out"], ref, bound, "attention of the step")
    for b, m in enumerate(lens):
        assert torch.allclose(d["acc"][b, :, :m].double().cpu(), p[b].view(2, 4, m).sum(1), rtol=1e-4, atol=1e-6)


def test_streams_graphs_and_repeats():
    """The same step eagerly, on another stream, and captured and replayed with eager work between: the
    same bits every time."""
    ref = _layer(5)
    ref["c"].dlen.copy_(_dev32([6, 41, 60]))
    _layer_step(ref)
    torch.cuda.synchronize()
    keys = ("qkv", "out", "lse", "acc", "y", "kept")

    def fresh():
        d = _layer(5)
        d["c"].dlen.copy_(_dev32([6, 41, 60]))
        return d

    d = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _layer_step(d, stream=s)
    s.synchronize()
    assert all(torch.equal(d[k], ref[k]) for k in keys) and torch.equal(d["c"].dk, ref["c"].dk)

    d = fresh()
    start = {k: d[k].clone() for k in ("acc",)}
    k0, v0, l0 = d["c"].dk.clone(), d["c"].dv.clone(), d["c"].dlen.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _layer_step(d)
    for _ in range(4):
        d["acc"].copy_(start["acc"])
        d["c"].dk.copy_(k0)
        d["c"].dv.copy_(v0)
        d["c"].dlen.copy_(l0)
        for k in ("out", "lse", "y", "kept"):
            d[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(d[k], ref[k]) for k in keys)
        assert torch.equal(d["c"].dk, ref["c"].dk) and torch.equal(d["c"].dlen, ref["c"].dlen)
        other = _layer(5)
        other["c"].dlen.copy_(_dev32([6, 41, 60]))
        _layer_step(other)
        assert all(torch.equal(other[k], ref[k]) for k in keys)


# ------------------------------------------------------------------ sizes that the small cases do not reach
def _many(batch, seed, most_q):
    """Row counts and lengths of many sequences: empty ones, ones without rows, ones with more rows than entries."""
    r = np.random.default_rng(seed)
    q = [int(v) for v in r.integers(0, most_q + 1, batch)]
    lens = [int(v) for v in r.choice([0, 1, 15, 16, 17, 40, 130, 301], batch)]
    q[-1], lens[-1] = 1, 33
    return q, lens


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch,most_q", [(65, 1), (130, 4), (300, 1), (70, 60)])
def test_many_sequences(batch, most_q, elem):
    q_len, lens = _many(batch, batch, most_q)
    Hq, Hkv, D, page = 8, 2, 64, 16
    c, start, q, scale, _ = _attn_case((Hq, Hkv, D, page, elem, 0, q_len, lens), 21)
    kv, _, out, lse = _run_attn(c, start, q, scale, 0)
    n = start[-1]
    ref, ref_lse, bound, p = R.attention(q, c, start, scale, 0)
    _within(out[:n], ref[:n], bound[:n], "attention")
    assert (out[n:] == 5).all() and (lse[n:] == 5).all()
    acc = torch.zeros(batch, Hkv, c.cols * page, device=DEV)
    oes.attn_weigh(q.to(DEV), lse.contiguous(), kv, _dev32(start), scale, acc)
    for b, m in enumerate(lens):
        add = p[b].view(p[b].shape[0], Hkv, Hq // Hkv, m).sum((0, 2))
        # as in test_attn_weigh, with the kernel's own lse: a score's error once more
        rel = 4 * ((D + 4) * R.U * 8 * math.sqrt(D) + 16 * R.U) + (max(1, p[b].shape[0] * 4) + 2) * R.U
        _within(acc[b, :, :m], add, rel * add + 1e-30, b)
        assert (acc[b, :, m:] == 0).all()
    # the rows' own k and v: entry len - rows + i gets row i, and no other entry changes
    k = torch.randn(n, Hkv, D, generator=_gen(2)).bfloat16()
    freq = torch.zeros(D // 2, dtype=torch.float64, device=DEV)
    oes.rope_append(q[:n].to(DEV), out[:n].contiguous(), k.to(DEV), k.to(DEV), freq, torch.arange(n, dtype=torch.int32, device=DEV), kv, _dev32(start))
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, (a, m) in enumerate(zip(q_len, lens)):
        for i in range(max(0, a - m), a):
            j, row = m - a + i, k[start[b] + i]
            pg, r = int(c.table[b, j // page]), j % page
            if elem == "bf16":
                want_k[pg, r], want_v[pg, r] = row, row
            else:
                want_k[pg, r] = (row.float() / torch.tensor(c.k_scale)).clamp(-448, 448).to(torch.float8_e4m3fn)
                want_v[pg, r] = (row.float() / torch.tensor(c.v_scale)).clamp(-448, 448).to(torch.float8_e4m3fn)
    bits = torch.int16 if elem == "bf16" else torch.uint8
    assert torch.equal(c.dk.cpu().view(bits), want_k.view(bits)) and torch.equal(c.dv.cpu().view(bits), want_v.view(bits))
    # and the eviction of all of them
    budget = 40
    kept = torch.empty(batch, Hkv, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(batch, dtype=torch.int32, device=DEV)
    ws = torch.empty(oes.kv_evict_workspace_bytes(kv, budget), dtype=torch.uint8, device=DEV)
    before = acc.cpu().clone()
    oes.kv_evict(kv, acc, budget, kept, new_len, ws, 4, 8)
    kv.check()
    assert torch.equal(kept.cpu(), R.evict(before, lens, c, budget, 4, 8))
    assert new_len.tolist() == [min(m, budget) for m in lens]


@pytest.mark.parametrize("case", [(8, 1, 128, 16, "bf16", 0, [1], [70001]), (4, 4, 64, 64, "e4m3", 0, [2, 1], [40003, 9]),
                                  (4, 2, 64, 1, "bf16", 0, [3, 1], [50, 190]), (2, 2, 128, 16, "bf16", 1000, [1, 1], [33333, 20])], ids=str)
def test_attn_long(case):
    """One row over many parts of a long cache, and pages of a single entry."""
    c, start, q, scale, window = _attn_case(case, 23, fill=None)
    kv, dq, out, lse = _run_attn(c, start, q, scale, window)
    n, Hq, Hkv = start[-1], case[0], case[1]
    ref, ref_lse, bound, p = R.attention(q, c, start, scale, window)
    _within(out[:n], ref[:n], bound[:n], case)
    acc = torch.zeros(len(c.lens), Hkv, c.cols * c.page, device=DEV)
    lse32 = ref_lse.float()
    oes.attn_weigh(dq.contiguous(), lse32.to(DEV), kv, _dev32(start), scale, acc, window)
    D = case[2]
    for b, m in enumerate(c.lens):
        add = p[b].view(p[b].shape[0], Hkv, Hq // Hkv, m).sum((0, 2))
        rel = 2 * ((D + 4) * R.U * 8 * math.sqrt(D) + 16 * R.U) + (p[b].shape[0] * Hq // Hkv + 2) * R.U
        _within(acc[b, :, :m], add, rel * add + 1e-30, (case, b))


@pytest.mark.parametrize("budget,first,last,lens", [(17000, 5, 100, [40000, 16384, 17001]), (60, 4, 10, [16385, 16384, 33000])])
def test_evict_long(budget, first, last, lens):
    """More entries than a workgroup holds in registers."""
    c = R.Cache(29, lens, 2, 16, 64)
    acc = torch.rand(len(lens), 2, c.cols * 64, generator=_gen(6))
    acc[:, :, 1::2] = (acc[:, :, 1::2] * 8).round() / 8
    kv, dacc = c.handle(oes), acc.to(DEV)
    kept = torch.empty(len(lens), 2, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(len(lens), dtype=torch.int32, device=DEV)
    ws = torch.empty(oes.kv_evict_workspace_bytes(kv, budget), dtype=torch.uint8, device=DEV)
    oes.kv_evict(kv, dacc, budget, kept, new_len, ws, first, last)
    kv.check()
    ref = R.evict(acc, lens, c, budget, first, last)
    assert torch.equal(kept.cpu(), ref) and new_len.tolist() == [min(m, budget) for m in lens]
    for b, m in enumerate(lens):
        if m > budget:
            for h in range(2):
                src, to = ref[b, h].long(), torch.arange(budget)
                assert torch.equal(c.dk.cpu()[c.table[b, to // 64].long(), to % 64, h], c.k[c.table[b, src // 64].long(), src % 64, h])
                assert torch.equal(dacc[b, h, :budget].cpu(), acc[b, h, src])


def test_cache_past_32_bits():
    """The same sequences in the first pages and in pages behind 2^32 elements: the same bits of every operator."""
    Hq, Hkv, D, page, lens, q_len = 16, 8, 128, 64, [200, 64, 1], [9, 1, 1]
    c = R.Cache(31, lens, Hkv, D, page)
    total = (1 << 32) // (page * Hkv * D) + c.pages + 3
    shift = total - c.pages
    start, n = _dev32(_starts(q_len)), sum(q_len)
    g = _gen(3)
    q, k, v = (torch.randn(n, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    freq, pos = torch.from_numpy(oes.rope_freqs(D)[0]).to(DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    got = []
    for at in (0, shift):
        dk, dv = (torch.empty(total if at else c.pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        dk[at:at + c.pages], dv[at:at + c.pages] = c.dk, c.dv
        kv = oes.KvPages(dk, dv, c.dtable + at, c.dlen)
        q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(n, Hq, device=DEV)
        acc = torch.zeros(3, Hkv, c.cols * page, device=DEV)
        kept, new_len = torch.empty(3, Hkv, 50, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
        oes.rope_append(q, q_out, k, v, freq, pos, kv, start)
        oes.attn(q_out, out, kv, start, D ** -0.5, torch.empty(oes.attn_workspace_bytes(kv, Hq, n), dtype=torch.uint8, device=DEV), lse=lse)
        oes.attn_weigh(q_out, lse, kv, start, D ** -0.5, acc)
        oes.kv_evict(kv, acc, 50, kept, new_len, torch.empty(oes.kv_evict_workspace_bytes(kv, 50), dtype=torch.uint8, device=DEV), 4, 8)
        kv.check()
        got.append((q_out, out, lse, acc, kept, new_len, dk[at:at + c.pages].clone(), dv[at:at + c.pages].clone()))
        del dk, dv, kv
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][4][0] >= 0).all()


def test_two_graphs_at_once():
    """Two captured steps of two layers, with workspaces of their own, replayed on two streams at the same time."""
    refs, layers, graphs, states = [], [], [], []
    for i in range(2):
        for into in (refs, layers):
            d = _layer(40 + i)
            d["c"].dlen.copy_(_dev32([6, 41 + i, 60]))
            into.append(d)
        _layer_step(refs[i])
        d = layers[i]
        states.append([d["acc"].clone(), d["c"].dk.clone(), d["c"].dv.clone(), d["c"].dlen.clone()])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            _layer_step(d)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for d, s in zip(layers, states):
            for to, x in zip((d["acc"], d["c"].dk, d["c"].dv, d["c"].dlen), s):
                to.copy_(x)
            for k in ("out", "lse", "y", "kept"):
                d[k].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for d, r in zip(layers, refs):
            assert all(torch.equal(d[k], r[k]) for k in ("qkv", "out", "lse", "acc", "y", "kept"))
            assert torch.equal(d["c"].dk, r["c"].dk) and torch.equal(d["c"].dv, r["c"].dv)

"""Decode steps of the whole attention half, each operator against its float64 reference on the state that it found,
over caches that earlier steps have cut; and sizes beyond the other tests': more tokens than rope has waves, tables far
wider than their sequences."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _dev32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _within(got, ref, bound, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


def _rope_bound(x, ref):
    """Half a bf16 step, and fp32: sine and cosine off by 2^-22 (4 U, of values up to mscale), two products and a sum."""
    mag = x.double().abs().amax(-1, keepdim=True) * 2 * 1.5
    return R.BF * ref.abs() + (1 + R.BF) * 8 * R.U * mag


def _weight_rel(D, rows):
    """Relative error of an entry's weight: twice a score's (D + 4) U of scale sum |q k| <= 8 sqrt(D), once for the weight
    and once for the kernel's own log-sum-exp, and the sum over the rows."""
    return 4 * ((D + 4) * R.U * 8 * math.sqrt(D) + 16 * R.U) + (rows + 2) * R.U


def _banks(fmt, N, K, seed):
    g = _gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    if fmt == "q4_0":
        return [codes, (0.01 * torch.randn(N, K // 32, generator=g)).half()]
    return [codes, torch.randint(0x30, 0x50, (N, K // 16), dtype=torch.uint8, generator=g), (1e-2 * torch.randn(N, generator=g)).half()]


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
def test_every_operator_of_every_decode_step(elem):
    H, Hq, Hkv, D, page, budget, first, last = 256, 8, 2, 64, 16, 48, 2, 8
    G, scale, lens = Hq // Hkv, D ** -0.5, [5, 40, 47]
    B = len(lens)
    c = R.Cache(81, [page * 4] * B, Hkv, D, page, elem)
    kv, cap = c.handle(oes), c.cols * page
    wq, wo = _banks("q4_0", (Hq + 2 * Hkv) * D, H, 82), _banks("nvfp4", H, Hq * D, 83)
    dwq, dwo = [b.to(DEV) for b in wq], [b.to(DEV) for b in wo]
    freq, m = oes.rope_freqs(D, 10000.0, "linear", 2.0)
    freq = torch.from_numpy(freq)
    x = torch.randn(B, H, generator=_gen(84)).bfloat16().to(DEV)
    pos, start, acc = _dev32(lens), _dev32(list(range(B + 1))), torch.zeros(B, Hkv, cap, device=DEV)
    kept, lse = torch.empty(B, Hkv, budget, dtype=torch.int32, device=DEV), torch.empty(B, Hq, device=DEV)
    out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(oes.attn_workspace_bytes(kv, Hq, B) + 16, dtype=torch.uint8, device=DEV)
    ews = torch.empty(oes.kv_evict_workspace_bytes(kv, budget), dtype=torch.uint8, device=DEV)
    bits = torch.int16 if elem == "bf16" else torch.uint8
    cuts = 0
    for step in range(8):
        lens = [n + 1 for n in lens]
        c.dlen.copy_(_dev32(lens))
        acc[torch.arange(B), :, torch.tensor(lens) - 1] = 0
        c.lens = lens

        qkv, y = torch.empty(B, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, dtype=torch.bfloat16, device=DEV)
        oes.linear("q4_0", x, dwq, qkv)
        _within(qkv, *R.linear("q4_0", x.cpu(), wq, qkv.shape[1]), (step, "q, k, v"))

        parts = qkv.view(B, Hq + 2 * Hkv, D)
        before = parts.cpu().clone()
        q, k, v = parts[:, :Hq], parts[:, Hq:Hq + Hkv], parts[:, Hq + Hkv:]
        k0, v0 = c.dk.cpu().contiguous(), c.dv.cpu().contiguous()
        oes.rope_append(q, q, k, v, freq.to(DEV), pos, kv, start, mscale=m)
        ref = R.turn(before[:, :Hq], pos, freq, m, "half", D)
        _within(q, ref, _rope_bound(before[:, :Hq], ref), (step, "rotated q"))
        new_k = R.turn(before[:, Hq:Hq + Hkv], pos, freq, m, "half", D)
        bound = _rope_bound(before[:, Hq:Hq + Hkv], new_k)
        k1, v1 = c.dk.cpu().contiguous(), c.dv.cpu().contiguous()
        for b, n in enumerate(lens):
            p, r = int(c.table[b, (n - 1) // page]), (n - 1) % page
            if elem == "bf16":
                _within(k1[p, r], new_k[b], bound[b], (step, "k"))
                assert torch.equal(v1[p, r], before[b, Hq + Hkv:])
            else:
                lo, hi = ((new_k[b] - bound[b]) / c.k_scale).clamp(-448, 448), ((new_k[b] + bound[b]) / c.k_scale).clamp(-448, 448)
                assert ((k1[p, r].double() >= R.to_e4m3(lo)) & (k1[p, r].double() <= R.to_e4m3(hi))).all()
                want = R.to_e4m3((before[b, Hq + Hkv:].float() / torch.tensor(c.v_scale)).double())
                assert torch.equal(v1[p, r].double(), want)
            k0[p, r], v0[p, r] = k1[p, r], v1[p, r]
        assert torch.equal(k0.view(bits), k1.view(bits)) and torch.equal(v0.view(bits), v1.view(bits)), (step, "another entry changed")

        oes.attn(q, out, kv, start, scale, ws, lse=lse)
        c.k, c.v = k1, v1
        ref, ref_lse, bound, p = R.attention(q.cpu(), c, list(range(B + 1)), scale)
        _within(out, ref, bound, (step, "attention"))
        _within(lse, ref_lse, (D + 4) * R.U * 8 * math.sqrt(D) + 8 * R.U * (1 + ref_lse.abs()), (step, "log-sum-exp"))

        acc0 = acc.cpu().clone()
        oes.attn_weigh(q, lse, kv, start, scale, acc)
        acc1, rel = acc.cpu(), _weight_rel(D, G)
        for b, n in enumerate(lens):
            add = p[b].view(Hkv, G, n).sum(1)
            want = acc0[b, :, :n].double() + add
            _within(acc1[b, :, :n], want, rel * add + 2 * R.U * want + 1e-30, (step, "weights"))
            assert torch.equal(acc1[b, :, n:], acc0[b, :, n:])
            # every query head's weights sum to one: G to a cache head (acc's rounding on top: 2 U of its values)
            got = (acc1[b, :, :n].double() - acc0[b, :, :n].double()).sum(1)
            assert ((got - G).abs() <= G * rel + 2 * R.U * want.sum(1)).all(), (step, got)

        oes.linear("nvfp4", out.view(B, -1), dwo, y)
        _within(y, *R.linear("nvfp4", out.view(B, -1).cpu(), wo, H), (step, "output projection"))

        oes.kv_evict(kv, acc, budget, kept, c.dlen, ews, first, last)
        kv.check()
        want = R.evict(acc1, lens, c, budget, first, last)
        assert torch.equal(kept.cpu(), want)
        a2 = acc1.clone()
        k2, v2 = k1.view(bits).clone(), v1.view(bits).clone()
        for b, n in enumerate(lens):
            if n <= budget:
                continue
            cuts += 1
            to = torch.arange(budget)
            for h in range(Hkv):
                src = want[b, h].long()
                for new, old in ((k2, k1.view(bits)), (v2, v1.view(bits))):
                    new[c.table[b, to // page].long(), to % page, h] = old[c.table[b, src // page].long(), src % page, h]
                a2[b, h, to] = acc1[b, h, src]
        assert torch.equal(c.dk.cpu().contiguous().view(bits), k2) and torch.equal(c.dv.cpu().contiguous().view(bits), v2)
        assert torch.equal(acc.cpu(), a2)
        lens = [min(n, budget) for n in lens]
        assert c.dlen.tolist() == lens
        x = (y.float() / (1e-3 + y.float().square().mean(-1, keepdim=True).sqrt())).bfloat16()
        pos += 1
    assert cuts >= 7


@pytest.mark.parametrize("layout,D,rot", [("half", 64, 64), ("interleaved", 64, 40), ("half", 48, 18)])
def test_rope_of_more_tokens_than_waves(layout, D, rot):
    """A wave takes several tokens, one after the other, through one table of sines and cosines."""
    n, heads, g = 8192 * 2 + 77, 3, _gen(91)
    freq, m = oes.rope_freqs(rot, 10000.0, "yarn", 4.0, 2048)
    freq = torch.from_numpy(freq)
    x, pos = torch.randn(n, heads, D, generator=g).bfloat16(), torch.randint(0, 1 << 20, (n,), generator=g).int()
    y = torch.full((n + 1, heads, D), 9.0, dtype=torch.bfloat16, device=DEV)
    oes.rope(x.to(DEV), y[:n], freq.to(DEV), pos.to(DEV), layout, m)
    ref = R.turn(x, pos, freq, m, layout, rot)
    _within(y[:n], ref, _rope_bound(x, ref), (layout, D, rot))
    assert (y[n] == 9).all()


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
def test_rope_append_of_more_tokens_than_waves(elem):
    q_len, lens, Hq, Hkv, D, page = [8200, 0, 700, 1], [8200, 5, 1000, 12], 2, 1, 64, 16
    c, n, g = R.Cache(92, lens, Hkv, D, page, elem), sum(q_len), _gen(93)
    start = [0]
    for a in q_len:
        start.append(start[-1] + a)
    freq = torch.from_numpy(oes.rope_freqs(D)[0])
    q, k, v = (torch.randn(n, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    pos = torch.arange(n, dtype=torch.int32)
    q_out, kv = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV), c.handle(oes)
    oes.rope_append(q.to(DEV), q_out, k.to(DEV), v.to(DEV), freq.to(DEV), pos.to(DEV), kv, _dev32(start))
    kv.check()
    ref = R.turn(q, pos, freq, 1.0, "half", D)
    _within(q_out, ref, _rope_bound(q, ref), "q")
    new_k = R.turn(k, pos, freq, 1.0, "half", D)
    bound, got_k, got_v = _rope_bound(k, new_k), c.dk.cpu().double(), c.dv.cpu().double()
    old_k, old_v = c.k.double(), c.v.double()
    for b, (a, e) in enumerate(zip(q_len, lens)):
        j, t = torch.arange(e - a, e), slice(start[b], start[b + 1])
        at = (c.table[b, j // page].long(), j % page)
        if elem == "bf16":
            _within(got_k[at], new_k[t], bound[t], "k")
            assert torch.equal(got_v[at], v[t].double())
        else:
            assert torch.equal(got_v[at], R.to_e4m3((v[t].float() / torch.tensor(c.v_scale)).double()))
            lo, hi = ((new_k[t] - bound[t]) / c.k_scale).clamp(-448, 448), ((new_k[t] + bound[t]) / c.k_scale).clamp(-448, 448)
            assert ((got_k[at] >= R.to_e4m3(lo)) & (got_k[at] <= R.to_e4m3(hi))).all()
        old_k[at], old_v[at] = got_k[at], got_v[at]
    assert torch.equal(old_k, got_k) and torch.equal(old_v, got_v), "another entry changed"


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,window,q_len,lens", [(8, 2, 64, 0, [100], [1500]), (4, 1, 128, 0, [90, 1, 40], [300, 900, 40]),
                                                        (8, 2, 64, 200, [60, 60], [800, 70]), (8, 2, 64, 0, [1, 1], [700, 3])], ids=str)
def test_tables_far_wider_than_their_sequences(Hq, Hkv, D, window, q_len, lens, elem):
    """Tables for 131072 entries, whose unused columns hold no page of the cache."""
    page = 16
    c = R.Cache(95, lens, Hkv, D, page, elem, cols=131072 // page, fill=math.nan)
    for b, n in enumerate(lens):
        c.table[b, -(-n // page):] = -5
    c.to(DEV)
    start = [0]
    for a in q_len:
        start.append(start[-1] + a)
    n, kv, scale = start[-1], c.handle(oes), D ** -0.5
    q = torch.randn(n, Hq, D, generator=_gen(96)).bfloat16()
    out, lse = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(n, Hq, device=DEV)
    ws = torch.full((oes.attn_workspace_bytes(kv, Hq, n) + 16,), 255, dtype=torch.uint8, device=DEV)
    oes.attn(q.to(DEV), out, kv, _dev32(start), scale, ws, window, lse)
    ref, ref_lse, bound, p = R.attention(q, c, start, scale, window)
    _within(out, ref, bound, "attention")
    _within(lse, ref_lse, (D + 4) * R.U * 8 * math.sqrt(D) + 8 * R.U * (1 + ref_lse.abs()), "log-sum-exp")
    acc = torch.zeros(len(lens), Hkv, 131072, device=DEV)
    oes.attn_weigh(q.to(DEV), lse, kv, _dev32(start), scale, acc, window)
    for b, m in enumerate(lens):
        add = p[b].view(p[b].shape[0], Hkv, Hq // Hkv, m).sum((0, 2))
        _within(acc[b, :, :m], add, _weight_rel(D, p[b].shape[0] * (Hq // Hkv)) * add + 1e-30, (b, "weights"))
        assert (acc[b, :, m:] == 0).all()
    kv.check()

"""attn_weigh where a product is not finite: a row that adds nothing (log-sum-exp -inf, or none at all) adds nothing
whatever its scores, and an infinite key whose scores are -inf receives 0."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _starts(q_len):
    start = [0]
    for a in q_len:
        start.append(start[-1] + a)
    return start, torch.tensor(start, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("Hq,Hkv,D,q_len,lens", [
    (12, 2, 64, [40], [300]),         # 6 heads a group: 126 of 128 rows of a tile are used, then a short tile
    (8, 2, 128, [50, 33], [200, 133]),
    (5, 1, 256, [60], [190]),
    (8, 2, 64, [1, 2], [300, 70]),    # decode
    (3, 3, 48, [1], [65])], ids=str)
def test_an_infinite_key_with_scores_of_minus_infinity_receives_nothing(Hq, Hkv, D, q_len, lens):
    c = R.Cache(61, lens, Hkv, D, 16)
    kv, scale = c.handle(oes), D ** -0.5
    start, dstart = _starts(q_len)
    q = torch.randn(start[-1], Hq, D, generator=torch.Generator().manual_seed(62)).bfloat16()
    q[..., 2] = -q[..., 2].abs().clamp(min=0.125)
    for b in range(len(lens)):
        c.dk[int(c.table[b, 0]), 3, :, 2] = math.inf     # entry 3: q . k = -inf for every row
    dq = q.to(DEV)
    out, lse = torch.empty_like(dq), torch.empty(start[-1], Hq, device=DEV)
    ws = torch.empty(oes.attn_workspace_bytes(kv, Hq, start[-1]) + 16, dtype=torch.uint8, device=DEV)
    oes.attn(dq, out, kv, dstart, scale, ws, lse=lse)
    acc = torch.rand(len(lens), Hkv, c.cols * 16, generator=torch.Generator().manual_seed(63))
    dacc = acc.to(DEV)
    oes.attn_weigh(dq, lse, kv, dstart, scale, dacc)
    assert torch.equal(dacc[:, :, 3].cpu(), acc[:, :, 3])
    # every other entry: against float64 (errors as derived for the plain tests, with the kernel's own lse)
    c.k = c.dk.cpu()
    _, _, _, p = R.attention(q, c, start, scale)
    for b, m in enumerate(lens):
        add = p[b].view(p[b].shape[0], Hkv, Hq // Hkv, m).sum((0, 2))
        rows = p[b].shape[0] * (Hq // Hkv)
        rel = 4 * ((D + 4) * R.U * 8 * math.sqrt(D) + 16 * R.U) + (rows + 2) * R.U
        ref = acc[b, :, :m].double() + add
        assert ((dacc[b, :, :m].double().cpu() - ref).abs() <= rel * add + 2 * R.U * ref + 1e-30).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,q_len,lens", [(8, 2, 64, [100], [300]), (12, 2, 128, [45], [200]),
                                                 (8, 2, 128, [1, 3], [300, 70]), (16, 1, 64, [30], [64])], ids=str)
def test_a_row_without_a_sum_adds_nothing(bad, elem, Hq, Hkv, D, q_len, lens):
    """lse = -inf rows with queries that are not finite: the weights are those of the other rows, to the bit of a
    call in which such rows hold ordinary queries."""
    c = R.Cache(65, lens, Hkv, D, 16, elem)
    kv, scale = c.handle(oes), D ** -0.5
    start, dstart = _starts(q_len)
    n = start[-1]
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(66)).bfloat16().to(DEV)
    lse = torch.full((n, Hq), 4.0, device=DEV)
    none = torch.zeros(n, Hq, dtype=torch.bool, device=DEV)
    none[0], none[n - 1, 1], none[n // 2, Hq - 1] = True, True, True
    lse[none] = -math.inf
    acc0, acc = (torch.zeros(len(lens), Hkv, c.cols * 16, device=DEV) for _ in range(2))
    oes.attn_weigh(q, lse, kv, dstart, scale, acc0)
    assert acc0.isfinite().all()
    q[none] = bad
    oes.attn_weigh(q, lse, kv, dstart, scale, acc)
    assert torch.equal(acc, acc0)


def test_rows_without_a_sum_hide_keys_that_are_not_finite():
    for elem, bad in (("bf16", math.inf), ("bf16", math.nan), ("e4m3", math.nan)):
        for q_len, m in ((100, 300), (2, 300)):
            c = R.Cache(67, [m], 2, 64, 16, elem)
            p = int(c.table[0, 0])
            if elem == "bf16":
                c.dk[p, 1] = bad
            else:
                c.dk.view(torch.uint8)[p, 1] = 0x7f
            q = torch.randn(q_len, 8, 64, generator=torch.Generator().manual_seed(68)).bfloat16().to(DEV)
            acc = torch.rand(1, 2, c.cols * 16, device=DEV)
            before = acc.clone()
            oes.attn_weigh(q, torch.full((q_len, 8), -math.inf, device=DEV), c.handle(oes),
                           torch.tensor([0, q_len], dtype=torch.int32, device=DEV), 0.125, acc)
            assert torch.equal(acc, before)

"""Attention rows whose scores are NaN: NaN in the output and the log-sum-exp, whichever way the row's parts are
joined, and every other row as without them."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _attn(q, kv, start, scale, window=0):
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    ws = torch.full((oes.attn_workspace_bytes(kv, q.shape[1], q.shape[0]) + 16,), 255, dtype=torch.uint8, device=DEV)
    oes.attn(q, out, kv, start, scale, ws, window, lse)
    return out, lse


# heads, kv_heads, D, page, elem, new tokens, entries
CASES = [
    (8, 2, 64, 16, "bf16", [1], [40]),                    # one token, entries of one workgroup
    (8, 2, 128, 16, "bf16", [1, 1, 2], [5000, 33, 700]),  # decode, rows shared by workgroups
    (8, 2, 128, 64, "e4m3", [1, 1], [3000, 90]),
    (4, 1, 256, 16, "bf16", [2], [900]),
    (8, 2, 64, 16, "bf16", [90, 40], [90, 200]),          # chunks, one part
    (8, 1, 128, 16, "bf16", [100], [4000]),               # a chunk whose entries are split
    (40, 1, 64, 32, "e4m3", [9], [3000]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_a_row_with_a_nan_query_is_nan(case):
    Hq, Hkv, D, page, elem, q_len, lens = case
    c = R.Cache(51, lens, Hkv, D, page, elem)
    kv, scale = c.handle(oes), D ** -0.5
    start = [0]
    for a in q_len:
        start.append(start[-1] + a)
    dstart = torch.tensor(start, dtype=torch.int32, device=DEV)
    n = start[-1]
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(52)).bfloat16().to(DEV)
    clean, lse0 = _attn(q, kv, dstart, scale)
    assert clean.isfinite().all() and lse0.isfinite().all()
    bad = torch.zeros(n, Hq, dtype=torch.bool, device=DEV)
    for i, t in enumerate({0, n // 2, n - 1}):
        bad[t, (3 * i) % Hq] = True
    q2 = q.clone()
    q2[..., D - 1][bad] = math.nan
    out, lse = _attn(q2, kv, dstart, scale)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], lse0[~bad])
    # and the weights of such a row are NaN, those that other cache heads receive as without it
    acc0, acc = (torch.zeros(len(lens), Hkv, c.cols * page, device=DEV) for _ in range(2))
    oes.attn_weigh(q, lse0, kv, dstart, scale, acc0)
    oes.attn_weigh(q2, lse, kv, dstart, scale, acc)
    for b, (a, m) in enumerate(zip(q_len, lens)):
        for g in range(Hkv):
            rows = bad[start[b]:start[b + 1], g * (Hq // Hkv):(g + 1) * (Hq // Hkv)].any(1).nonzero().flatten().tolist()
            seen = m - a + max(rows) + 1 if rows else 0   # entries that the last such row sees
            assert acc[b, g, :seen].isnan().all()
            assert torch.equal(acc[b, g, seen:], acc0[b, g, seen:])


@pytest.mark.parametrize("elem", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len,lens", [([1, 1], [1, 300]), ([1, 1], [3000, 4000]), ([70, 1], [70, 9]), ([150], [4000])], ids=str)
def test_a_sequence_of_nan_keys_is_nan(elem, q_len, lens):
    """All keys of the first sequence NaN (one key, or many): its rows are NaN, another sequence's are not."""
    Hq, Hkv, D, page = 8, 2, 64, 16
    c = R.Cache(53, lens, Hkv, D, page, elem)
    start = [0, q_len[0]] + ([q_len[0] + q_len[1]] if len(q_len) > 1 else [])
    dstart = torch.tensor(start, dtype=torch.int32, device=DEV)
    q = torch.randn(start[-1], Hq, D, generator=torch.Generator().manual_seed(54)).bfloat16().to(DEV)
    clean, lse0 = _attn(q, c.handle(oes), dstart, 0.125)
    for p in c.table[0, :-(-lens[0] // page)].tolist():
        if elem == "bf16":
            c.dk[p, :, :, 7] = math.nan
        else:
            c.dk.view(torch.uint8)[p, :, :, 7] = 0x7f
    out, lse = _attn(q, c.handle(oes), dstart, 0.125)
    a = q_len[0]
    assert out[:a].isnan().all() and lse[:a].isnan().all()
    assert torch.equal(out[a:], clean[a:]) and torch.equal(lse[a:], lse0[a:])


@pytest.mark.parametrize("q_len,lens", [([1], [40]), ([1, 1], [3000, 90]), ([70], [70]), ([150], [4000])], ids=str)
def test_infinite_scores(q_len, lens):
    """Scores of -inf alone: as for a row that sees nothing.  +inf among them: NaN."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    c = R.Cache(55, lens, Hkv, D, page)
    c.dk[..., 0] = c.dk[..., 0].abs().clamp(min=0.125)
    start = [0]
    for a in q_len:
        start.append(start[-1] + a)
    dstart = torch.tensor(start, dtype=torch.int32, device=DEV)
    q = torch.randn(start[-1], Hq, D, generator=torch.Generator().manual_seed(56)).bfloat16().to(DEV)
    clean, lse0 = _attn(q, c.handle(oes), dstart, 0.125)
    q[-1, 0, 0], q[-1, 1, 0] = -math.inf, math.inf
    out, lse = _attn(q, c.handle(oes), dstart, 0.125)
    assert (out[-1, 0] == 0).all() and lse[-1, 0] == -math.inf
    assert out[-1, 1].isnan().all() and lse[-1, 1].isnan()
    out[-1, :2], lse[-1, :2] = clean[-1, :2], lse0[-1, :2]
    assert torch.equal(out, clean) and torch.equal(lse, lse0)

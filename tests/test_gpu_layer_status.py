"""KvPages.check() with calls on other streams than the current one: it sees what they met, and what it clears is gone
for good."""
import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 40_000_000   # cycles that a stream is kept busy for: some 20 ms


def _call(kv, c, stream=None):
    q, out = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    ws = torch.empty(oes.attn_workspace_bytes(kv, 4, 1) + 16, dtype=torch.uint8, device=DEV)
    torch.cuda.current_stream().synchronize()
    return (lambda: oes.attn(q, out, kv, start, 0.125, ws, stream=stream)), (q, out, start, ws)


def _cache(bad=True):
    c = R.Cache(71, [40], 2, 64, 16)
    if bad:
        c.table[0, 1] = -1
        c.to(DEV)
    return c


def test_check_waits_for_calls_on_other_streams():
    c = _cache()
    kv, s = c.handle(oes), torch.cuda.Stream()
    call, keep = _call(kv, c, s)
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        call()
        with pytest.raises(oes.OesError) as e:
            kv.check()
        assert e.value.status == oes.ERR_ARG
        kv.check()   # cleared, and nothing arrives later
    del keep


def test_what_a_check_clears_does_not_reach_a_later_call():
    """The current stream is busy when check() clears the word; a call on another stream right behind it is seen."""
    c = _cache()
    kv, s = c.handle(oes), torch.cuda.Stream()
    call, keep = _call(kv, c, s)
    for _ in range(3):
        call()
        torch.cuda._sleep(BUSY)
        with pytest.raises(oes.OesError):
            kv.check()
        call()
        s.synchronize()
        with pytest.raises(oes.OesError):
            kv.check()
    del keep


def test_a_handle_made_on_a_busy_stream_serves_another_at_once():
    """The word's first value comes from the constructor's stream: a call on another stream is not overwritten by it."""
    c = _cache()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = c.handle(oes)
    _, (q, out, start, ws) = _call(first, c)
    for _ in range(3):
        torch.cuda._sleep(BUSY)
        kv = c.handle(oes)
        oes.attn(q, out, kv, start, 0.125, ws, stream=s)
        with pytest.raises(oes.OesError):
            kv.check()
    good = _cache(bad=False).handle(oes)
    torch.cuda._sleep(BUSY)
    oes.attn(q, out, good, start, 0.125, ws, stream=s)
    good.check()


def test_a_handle_made_on_a_busy_side_stream_serves_the_default_one_at_once():
    c = _cache()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _, (q, out, start, ws) = _call(c.handle(oes), c)
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
            kv = c.handle(oes)
        oes.attn(q, out, kv, start, 0.125, ws)
        with pytest.raises(oes.OesError):
            kv.check()


def test_handles_in_captured_graphs():
    """A handle that is older than the capture, replayed between eager calls of another stream and checks."""
    c = _cache()
    kv, s = c.handle(oes), torch.cuda.Stream()
    call, keep = _call(kv, c)
    side, keep2 = _call(kv, c, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kv.check()
    for _ in range(3):
        graph.replay()
        with pytest.raises(oes.OesError):
            kv.check()
        kv.check()
        side()
        with pytest.raises(oes.OesError):
            kv.check()
    del keep, keep2

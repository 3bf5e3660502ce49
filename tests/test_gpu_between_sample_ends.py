"""Sampling at the ends of its range: uniform numbers of 0, -0 and from 1 on, entries that weigh nothing, and batches
that shrink."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests.test_gpu_between_ops import BF16, F32, _check_sample, _gen, _logits, _sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [8, 1000, 40000, 131072])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_negative_zero_is_zero(V, dtype):
    g, u = _gen(V), [-0.0, 0.0, -0.0, -1e-40, -math.inf]
    flat = torch.full((len(u), V), 3.25, dtype=dtype)
    flat[:, :3] = -math.inf
    for logits in (flat, _logits(g, len(u), V, dtype)):
        for s in ((None, None, None, None), (1.0, 5, 1.0, 0.0), (0.5, 0, 0.5, 0.0), (2.0, V // 2, 0.25, 0.5)):
            _check_sample(logits, u, *s)


@pytest.mark.parametrize("settings", [(None, None, None, None), (1.0, "most", 1.0, 0.0), (2.0, 0, 1.0, 0.0)],
                         ids=["none", "top-k", "twice as hot"])
@pytest.mark.parametrize("first", [0, 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_entries_that_weigh_nothing(settings, first, dtype):
    """Stretches of entries below 2^-44 of the largest, whose sum would weigh something, before, between and behind the
    others: they are never chosen, and the first and the last token are those of the others.  Stretches just above
    2^-44, whose entries each count as more than they weigh, end with their last entry."""
    g, V = _gen(7 + first), 60011
    t = 2.0 if settings[0] == 2.0 else 1.0
    nothing, little = -31.0 * t, -30.375 * t    # e^-31 = 3.4e-14, 2^-44 = 5.7e-14, e^-30.375 = 6.4e-14
    rows = torch.full((4, V), nothing)
    rows[0, 9000:9003] = torch.tensor([-1.0, -3.0, -0.5])
    rows[0, 30000] = 0.0
    rows[1, 20000:45000] = _logits(g, 1, 25000, F32)[0] / 4
    rows[2, 25000], rows[2, 50000:] = 0.0, little
    rows[3, 100], rows[3, 20000], rows[3, 33000:33005], rows[3, 58000] = -2.0, 0.0, little, -2.5
    rows[1] -= rows[1].max()
    rows[1, :20000], rows[1, 45000:] = nothing, nothing
    wide = torch.full((4, V + first), 50.0, dtype=dtype, device="cuda:0")
    wide[:, first:] = rows.to(dtype).to("cuda:0")
    t_, k, p, m = settings
    k = V - 100 if k == "most" else k
    for u in (0.0, 2.0 ** -24, 1.0, 3.0):
        _check_sample(wide[:, first:], [u] * 4, t_, k, p, m)
        ids, lp = _sample(wide[:, first:], [u] * 4, t_, k, p, m)
        # a smallest weight that everything which counts passes: weighed by another way, the same tokens
        again, lp2 = _sample(wide[:, first:], [u] * 4, t_, k, p, 1e-20)
        assert torch.equal(ids, again) and ((lp - lp2).abs() <= 2.0 ** -23 * lp.abs() + 1e-8).all()


@pytest.mark.parametrize("V", [100003, 128256])
def test_a_batch_that_shrinks_keeps_its_workspace(V):
    """The workspace of the largest batch, made once, through batches around the change of the slices' length."""
    g, most = _gen(V), 96
    logits, u = _logits(g, most, V, BF16).to("cuda:0"), torch.rand(most, generator=g).to("cuda:0")
    held = torch.empty(oes.sample_workspace_bytes(most, V), dtype=torch.uint8, device="cuda:0")
    k, p = torch.full((most,), 64, dtype=torch.int32, device="cuda:0"), torch.full((most,), 0.95, device="cuda:0")
    for n in (96, 82, 81, 80, 65, 64, 63, 1):
        ids = torch.full((most,), -7, dtype=torch.int32, device="cuda:0")
        oes.sample(logits[:n], u[:n], ids[:n], held, top_k=k[:n], top_p=p[:n])
        want, _ = _sample(logits[:n], u[:n].cpu(), None, 64, 0.95)
        assert torch.equal(ids[:n].cpu(), want) and (ids[n:] == -7).all(), n

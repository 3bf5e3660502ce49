"""Sigmoids of far negative values: as the formula down to 2^-126, and 0 (or the formula's value) below."""
import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests.test_gpu_between_ops import BF16, DEV, F32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
V = torch.tensor([-20.0, -60.0, -80.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -92.0, -104.0, -300.0, -1e30]).bfloat16()


def _near(got, v, act):
    """exp of an argument rounded to fp32 is off by |v| U, four more steps; what counts as 0 is below 2^-126, times |v| for silu."""
    got, v = got.double().cpu(), v.double()
    want = torch.exp(v) / (1 + torch.exp(v)) * (v if act == "silu" else 1)
    lost = torch.where(v < -87.3, 2.0 ** -126 * (v.abs() if act == "silu" else 1), 0.0)
    assert ((got - want).abs() <= want.abs() * (v.abs() + 4) * 4 * U + lost).all(), (act, got, want)
    assert (got[v < -104] == 0).all()


@pytest.mark.parametrize("n", [1, len(V)])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_products(n, act):
    for v in (V,) if n > 1 else V.split(1):
        x = torch.zeros(n, 8, dtype=BF16, device=DEV)
        x[:, 0] = v.to(DEV)
        w = torch.zeros(3, 8, dtype=BF16, device=DEV)
        w[:, 0] = 1
        y = torch.empty(n, 3, dtype=F32, device=DEV)
        oes.linear_bf16(x, w, y, act=act)
        for c in range(3):
            _near(y[:, c], v, act)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("shared", [False, True])
def test_gates(act, shared):
    n = len(V)
    x = torch.ones(n, 64, dtype=BF16, device=DEV)
    gate = V.to(DEV)[:, None] if shared else V.to(DEV)[:, None].expand(n, 64).contiguous()
    r = torch.empty(n, 64, dtype=F32, device=DEV)
    oes.norm(x, gate=gate, gate_act=act, res_out=r)
    for c in (0, 63):
        _near(r[:, c], V, act)

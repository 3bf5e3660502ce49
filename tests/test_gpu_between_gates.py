"""Norms with a gate per column on rows that leave lanes without columns: whatever an earlier call left
in those lanes' registers, the norm behind the gate is that of the row alone."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import between_ref as R
from tests.test_gpu_between_ops import BF16, DEV, F32, _gen, _randn, _spec, _within

pytestmark = pytest.mark.gpu

# (width that fills the lanes, widths of the same kernel that do not)
WIDTHS = [(32, (24,)), (64, (40, 56)), (128, (72, 96)), (256, (136, 160, 192)), (512, (264, 504)), (2048, (520, 768, 1032)),
          (4096, (2056, 2304, 2560, 2880, 3584)), (8192, (4104, 4608, 5376)), (16384, (8200, 12296))]


def _leave(n, heads, dim, x_kind, res_kind, fill):
    """Fills the gate's registers of every lane, all over the card, by calls of a full width."""
    shape = (n, heads, dim)
    x = torch.ones(shape, dtype=x_kind, device=DEV)
    res = None if res_kind is None else torch.ones(shape, dtype=res_kind, device=DEV)
    gate, y = torch.full(shape, fill, dtype=BF16, device=DEV), torch.empty(shape, dtype=BF16, device=DEV)
    for _ in range(3):
        oes.norm(x, y, pre=oes.Norm(), gate=gate, res=res)


@pytest.mark.parametrize("full,dims", WIDTHS, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("act,fill", [("plain", math.nan), ("plain", math.inf), ("sigmoid", math.nan), ("silu", -math.inf)])
@pytest.mark.parametrize("x_kind,res_kind", [(BF16, None), (BF16, F32), (F32, F32)])
def test_gates_per_column_behind_the_rows_end(full, dims, act, fill, x_kind, res_kind):
    # enough rows that every CU has held several
    n = max(2048, (1 << 21) // full)
    for dim in dims:
        g = _gen(dim)
        some = 65
        x, gate = _randn(g, some, 1, dim).to(x_kind), _randn(g, some, 1, dim, std=2.0).bfloat16()
        res = None if res_kind is None else _randn(g, some, 1, dim).to(res_kind)
        pre, pre_r = _spec(g, "rms", dim, BF16)
        post, post_r = _spec(g, "layer", dim, BF16)
        for post_, post_r_ in ((None, None), (post, post_r)):
            r, err = R.norm(x, post_r_, gate, act, 0.5, res)
            want, err = R.normed(r, err, pre_r)
            y = torch.empty(x.shape, dtype=BF16, device=DEV)
            xs, gs, rs = x.to(DEV), gate.to(DEV), None if res is None else res.to(DEV)
            torch.cuda.synchronize()
            _leave(n, 1, full, x_kind, res_kind, fill)
            oes.norm(xs, y, pre=pre, post=post_, gate=gs, gate_act=act, scale=0.5, res=rs)
            assert y.isfinite().all(), (dim, act, "columns behind the row's end took part")
            _within(y, want, R.stored(want, err, BF16), (dim, act))

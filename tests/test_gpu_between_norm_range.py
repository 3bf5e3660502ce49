"""Layer norms of rows whose sums or differences pass fp32: a finite row has a norm of 0, one with an infinity or
a NaN is NaN, and rows beside them are as ever."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import between_ref as R
from tests.test_gpu_between_ops import BF16, DEV, F32, _gen, _randn, _spec, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [8, 24, 64, 520, 1024, 2048, 2880, 8192, 8200, 16384])
@pytest.mark.parametrize("x_kind", [BF16, F32])
@pytest.mark.parametrize("side", ["pre", "post"])
def test_layer_norm_of_rows_beyond_fp32(dim, x_kind, side):
    g = _gen(dim)
    most = torch.finfo(x_kind).max
    x = _randn(g, 12, dim).to(x_kind)
    x[1] = 2.0 ** 120                                          # the sum overflows, the mean does not
    x[1, 0] = 2.0 ** 121
    x[2] = most
    x[2, 0] = most / 2
    x[3], x[3, ::2] = -most, most                              # differences of up to twice the largest
    x[4], x[4, 0] = -most, most
    x[5], x[5, dim - 1] = 2.0 ** 100, -2.0 ** 100              # squares beyond fp32
    x[6], x[6, dim // 2] = most, math.inf
    x[7, 0], x[8, dim - 1], x[9, 1] = -math.inf, math.nan, math.inf
    x[9, 2] = -math.inf
    own, spec = _spec(g, "layer", dim, F32, eps=1e-5)
    y = torch.empty(12, dim, dtype=BF16, device=DEV)
    oes.norm(x.to(DEV), y, **{side: own})
    bias = spec["b"].to(BF16)
    for row in (1, 2, 3, 4, 5):
        assert torch.equal(y[row].cpu(), bias), row
    assert y[6:10].isnan().all()
    rows = [0, 10, 11]
    want, err = R.normed(x[rows].double(), torch.zeros(3, dim, dtype=torch.float64), spec)
    _within(y[rows], want, R.stored(want, err, BF16), "rows")

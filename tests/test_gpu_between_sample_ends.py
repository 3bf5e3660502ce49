"""Sampling at the ends of its range: uniform numbers of 0, -0 and from 1 on."""
import math

import pytest
import torch

from tests.test_gpu_between_ops import BF16, F32, _check_sample, _gen, _logits

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

"""q4_0 linear over the whole range of bf16 activations: infinite ones give the product's infinities, and finite ones
of any size the product, in every way the work is split."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes
from tests import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MOST = torch.finfo(torch.bfloat16).max


def _q4_0(N, K, seed, low=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    if low:   # codes of one value in all rows
        codes[:] = low * 17
    return [codes, (1e-3 + 0.01 * torch.rand(N, K // 32, generator=g)).half()]


def _run(x, banks, N):
    y = torch.empty(x.shape[0], N, dtype=torch.bfloat16, device=DEV)
    oes.linear("q4_0", x.to(DEV), [b.to(DEV) for b in banks], y)
    return y.cpu()


# every split of the work: eight, four and two waves on K, one; x whole and in pieces; one, two and four tiles of tokens
SHAPES = [(1, 40, 256), (3, 100, 96), (2, 513, 2048), (1, 5003, 4128), (17, 5003, 288), (2, 9999, 2912), (2, 20005, 2080),
          (16, 24577, 1536), (20, 24600, 800), (40, 24593, 800), (70, 24611, 256), (5, 64, 7168)]


@pytest.mark.parametrize("n,N,K", SHAPES)
def test_large_activations(n, N, K):
    """One activation of every second token at the end of the range (each product of it with a weight stays within)."""
    banks = _q4_0(N, K, N + K)
    x = torch.randn(n, K, generator=torch.Generator().manual_seed(K)).bfloat16()
    for t in range(0, n, 2):
        x[t, (37 * t + K - 1 - (t % 5) * 61) % K] = MOST if t % 4 else -MOST
    y = _run(x, banks, N)
    ref, bound = R.linear("q4_0", x, banks, N)   # |w| <= 8 * 0.011: below 3e37
    bad = ~((y.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), y[bad][:3].tolist(), ref[bad][:3].tolist())


@pytest.mark.parametrize("code", [1, 15])
def test_blocks_of_the_largest_activations(code):
    """A whole block of activations at the end of the range, all of one sign: 32 * 8 * 3.4e38 before the scale, finite
    after it."""
    N, K = 40, 64
    banks = _q4_0(N, K, 3, code)
    banks[1][:] = 2.0 ** -10
    x = torch.zeros(2, K, dtype=torch.bfloat16)
    x[0, :32], x[1, 32:] = MOST, -MOST
    y = _run(x, banks, N)
    ref, bound = R.linear("q4_0", x, banks, N)
    assert ((y.double() - ref).abs() <= bound).all() and ref.abs().max() > 1e37


@pytest.mark.parametrize("n,N,K", SHAPES)
def test_infinite_activations(n, N, K):
    """Products with an infinite activation: infinite of the product's sign, NaN where the weight is 0 or two of them
    meet; a NaN activation gives NaN; the other tokens as ever."""
    banks = _q4_0(N, K, N - K)
    x = torch.randn(n, K, generator=torch.Generator().manual_seed(K + 1)).bfloat16()
    x[0, K // 2] = math.inf
    if n > 2:
        x[2, 1], x[2, K - 1] = -math.inf, -math.inf
        x[1, 5] = math.nan
    y = _run(x, banks, N)
    odd = ~x.isfinite().all(1)
    w = R.weights("q4_0", banks, N, K)
    for t in odd.nonzero().flatten().tolist():
        ref = (x[t].double() * w).sum(1)     # inf * w by IEEE arithmetic
        assert torch.equal(y[t].double().nan_to_num(7, math.inf, -math.inf), ref.nan_to_num(7, math.inf, -math.inf)), t
    ref, bound = R.linear("q4_0", x[~odd], banks, N)
    assert ((y[~odd].double() - ref).abs() <= bound).all()

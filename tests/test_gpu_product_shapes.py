"""The bf16 product at sizes that take each of its shapes through its main loop, against float64."""
import pytest

from tests.product_shapes import CASES
from tests.test_gpu_between_ops import BF16, F32, _check_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,N,K,act", CASES)
def test_main_loops(n, N, K, act):
    _check_product(n, N, K, act=act, pad=3)
    _check_product(n, N, K, act=act if act == "swiglu" else "gelu", bias=True, res=True, out=F32, scale=-0.5, wpad=8, seed=1)
    _check_product(n, N, K, act=act, res=True, scale=0.25, inplace=True, seed=2)

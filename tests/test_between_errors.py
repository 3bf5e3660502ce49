"""What the binding of the operators between the blocks refuses by itself: always an OesError that names the argument (CPU)."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes


def refused(call, *words):
    with pytest.raises(oes.OesError) as e:
        call()
    assert e.value.status == oes.ERR_ARG
    assert all(w in str(e.value) for w in words), str(e.value)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("act", ["relu", "", None, 3, -1, 2.0, 1 << 32])
def test_names_of_gates(act):
    x = bf(3, 64)
    refused(lambda: oes.norm(x, bf(3, 64), gate=bf(3, 64), gate_act=act), "gate_act", repr(act), "silu")


@pytest.mark.parametrize("act", ["relu", "SILU", None, 5, -1, 1.5, 1 << 32])
def test_names_of_activations(act):
    refused(lambda: oes.linear_bf16(bf(3, 64), bf(10, 64), bf(3, 10), act=act), "act", repr(act), "swiglu")


@pytest.mark.parametrize("kind", ["foo", None, 2, 1 << 32, 0.5])
def test_kinds_of_norms(kind):
    refused(lambda: oes.Norm(bf(64), kind=kind), "kind", repr(kind), "layer")


@pytest.mark.parametrize("value", [1e40, -1e39, math.inf, math.nan, 10 ** 400, "1", "x", None, [1.0], torch.zeros(2)], ids=str)
def test_numbers(value):
    x = bf(3, 64)
    refused(lambda: oes.norm(x, bf(3, 64), scale=value), "scale", repr(value))
    refused(lambda: oes.linear_bf16(x, bf(10, 64), bf(3, 10), scale=value), "scale")
    refused(lambda: oes.Norm(bf(64), eps=value), "eps")
    refused(lambda: oes.Norm(bf(64), offset=value), "offset")


def test_values_that_stay():
    """Numbers of the C enums, and whatever is a float, pass as before (to the refusal of tensors that are on no GPU)."""
    x = bf(3, 64)
    for a in (0, 1, 2, "plain", "sigmoid", "silu"):
        refused(lambda: oes.norm(x, bf(3, 64), gate=x, gate_act=a, scale=2), "not on a GPU")
    for a in (0, 1, 2, 3, "none", "sigmoid", "silu", "gelu"):
        refused(lambda: oes.linear_bf16(x, bf(10, 64), bf(3, 10), act=a, scale=torch.tensor(0.5)), "not on a GPU")
    refused(lambda: oes.linear_bf16(x, bf(20, 64), bf(3, 10), act=4), "not on a GPU")
    assert oes.Norm(bf(64), kind=1)._spec.kind == 1 and oes.Norm(bf(64), eps=0)._spec.eps == 0

"""What the binding of the operators between the blocks refuses by itself: always an OesError that names the argument (CPU)."""
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes


def refused(call, *words, status=oes.ERR_ARG):
    with pytest.raises(oes.OesError) as e:
        call()
    assert e.value.status == status
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


def test_sizes_beyond_the_c_interface():
    """Sizes that an int32 does not hold are refused as such, not cut to their low bits (rows of stride 0 take no memory)."""
    def rows(n, cols, kind=torch.bfloat16):
        return torch.zeros(1, cols, dtype=kind).expand(n, cols)

    def wide(n, cols, kind=torch.bfloat16):
        return torch.zeros(1, 1, dtype=kind).expand(n, cols)

    def beyond(call):
        refused(call, "too large", status=oes.ERR_UNSUPPORTED)

    for n in (1 << 31, (1 << 32) + 1):
        refused(lambda: oes.norm(rows(n, 64), rows(n, 64)), "too large")
        beyond(lambda: oes.linear_bf16(rows(n, 64), bf(10, 64), rows(n, 10)))
        beyond(lambda: oes.linear_bf16(bf(3, 64), rows(n, 64), wide(3, n)))
        beyond(lambda: oes.linear_bf16(wide(3, n), wide(10, n), bf(3, 10)))
        beyond(lambda: oes.sample(rows(n, 50), wide(1, n, torch.float32)[0], wide(1, n, torch.int32)[0], bf(0)))
        beyond(lambda: oes.sample(wide(3, n), torch.zeros(3), torch.zeros(3, dtype=torch.int32), bf(0)))
        beyond(lambda: oes.sample_workspace_bytes(n, 100))
        beyond(lambda: oes.sample_workspace_bytes(3, n))
    beyond(lambda: oes.sample_workspace_bytes(-(1 << 32) + 3, 100))
    beyond(lambda: oes.linear_bf16(bf(1, 64), rows(1 << 32, 64), wide(1, 1 << 31), act="swiglu"))

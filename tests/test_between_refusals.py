"""CPU checks of the operators between the blocks: refusals of the C ABI and of the binding
before any GPU work, and the layout that the binding packs."""
import ctypes
import math

import pytest
import torch

import offloaded_expert_slot_amd as oes

A = 1 << 12  # an aligned address that is never dereferenced: refusals happen before


def spec(**over):
    c = dict(w=A, b=0, kind=0, elem=oes.ELEM_BF16, eps=1e-6, offset=0.0)
    c.update(over)
    return oes.NormSpec(*[c[f] for f, _ in oes.NormSpec._fields_])


def norm(pre=None, post=None, **over):
    pre = spec() if pre is None else pre
    c = dict(post=0 if post is None else ctypes.addressof(post), pre=ctypes.addressof(pre) if pre else 0, x=A, gate=0,
             res=2 * A, res_out=3 * A, y=4 * A, x_row=128, x_head=64, gate_row=0, gate_head=0, gate_col=0, res_row=128,
             res_head=64, ro_row=128, ro_head=64, y_row=128, y_head=64, n=5, heads=2, dim=64, x_elem=oes.ELEM_BF16,
             res_elem=oes.ELEM_BF16, gate_act=0, scale=1.0, reserved=0)
    c.update(over)
    args = oes.NormArgs(*[c[f] for f, _ in oes.NormArgs._fields_])
    return oes.lib().oes_norm(ctypes.byref(args), None)


NORM_BAD = [dict(n=-1), dict(heads=0), dict(n=1 << 30, heads=4), dict(dim=0), dict(dim=60), dict(dim=16392), dict(dim=-8),
            dict(reserved=1), dict(x=0), dict(x=A + 8), dict(x_row=124), dict(x_row=-128), dict(x_head=60), dict(res=A + 4),
            dict(res_row=4), dict(ro_row=56), dict(ro_head=32), dict(res_out=3 * A + 2), dict(y=4 * A + 8), dict(y_row=32),
            dict(y_head=56), dict(res_out=0, y=0), dict(y=0), dict(scale=math.nan), dict(scale=math.inf), dict(res_out=A),
            dict(res_out=4 * A), dict(res_out=2 * A, ro_row=256), dict(y=A, y_row=256), dict(y=A, y_head=128),
            dict(y=2 * A), dict(gate=5 * A, gate_act=3), dict(gate=5 * A, gate_act=-1), dict(gate=5 * A, gate_col=2),
            dict(gate=5 * A, gate_row=-8), dict(gate=5 * A + 2, gate_col=1), dict(gate=5 * A, gate_col=1, gate_row=4),
            dict(gate=5 * A + 1), dict(gate=4 * A, gate_col=1), dict(gate=3 * A, gate_col=1),
            dict(x_elem=oes.ELEM_F32, y=A, x_row=128)]


@pytest.mark.parametrize("bad", NORM_BAD, ids=str)
def test_norm_refuses(bad):
    assert norm(**bad) == oes.ERR_ARG
    assert oes.lib().oes_last_error()


def test_norm_refuses_types_and_specs():
    assert norm(x_elem=oes.ELEM_FP16) == norm(res_elem=oes.ELEM_E4M3) == oes.ERR_UNSUPPORTED
    assert norm(pre=spec(elem=oes.ELEM_FP16)) == oes.ERR_UNSUPPORTED
    for bad in (dict(kind=2), dict(kind=-1), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(offset=math.inf),
                dict(w=A + 2), dict(b=A + 8)):
        assert norm(pre=spec(**bad)) == norm(post=spec(**bad)) == oes.ERR_ARG, bad
    assert oes.lib().oes_norm(None, None) == oes.ERR_ARG
    assert norm(n=0, x=0, res=0, res_out=3 * A, y=4 * A) == oes.OK


def test_packed_arguments_have_the_layout_of_the_struct():
    values = list(range(1, len(oes.NormArgs._fields_) + 1))
    packed = oes._NORM_ARGS.pack(*values)
    assert len(packed) == ctypes.sizeof(oes.NormArgs)
    back = oes.NormArgs.from_buffer_copy(packed)
    assert [getattr(back, f) for f, _ in oes.NormArgs._fields_] == values


def product(w=A, w_row=64, bias=0, N=10, K=64, x=2 * A, x_row=64, n=3, act=0, scale=1.0, res=0, res_row=10, y=3 * A,
            y_row=10, y_elem=oes.ELEM_BF16):
    return oes.lib().oes_linear_bf16(w, w_row, bias, N, K, x, x_row, n, act, scale, res, res_row, y, y_row, y_elem, None)


def test_product_refuses():
    for bad in (dict(N=0), dict(K=0), dict(K=60), dict(K=(1 << 20) + 8), dict(n=-1), dict(act=-1), dict(act=5),
                dict(scale=math.nan), dict(scale=-math.inf), dict(w=0), dict(x=0), dict(y=0), dict(w=A + 8), dict(x=A + 2),
                dict(w_row=60), dict(x_row=72 + 4), dict(bias=A + 1), dict(y=3 * A + 1), dict(res=A + 1), dict(w_row=56),
                dict(x_row=56), dict(y_row=9), dict(res=4 * A, res_row=9), dict(w_row=-64), dict(x_row=-64), dict(y_row=-10),
                dict(res=3 * A, res_row=12), dict(y=2 * A), dict(y=A), dict(bias=3 * A), dict(act=4, N=1, w_row=0),
                dict(y_elem=oes.ELEM_F32, y=3 * A + 2)):
        assert product(**bad) == oes.ERR_ARG, bad
    for bad in (dict(N=(1 << 22) + 1, y_row=1 << 23), dict(n=(1 << 19) + 1), dict(y_elem=oes.ELEM_FP16)):
        assert product(**bad) == oes.ERR_UNSUPPORTED, bad
    assert product(n=0, w=0, x=0, y=0) == oes.OK
    # more workgroups than a launch holds
    assert product(N=1 << 22, n=1 << 19, act=4, y_row=1 << 22) == oes.ERR_UNSUPPORTED


def sample(logits=A, elem=oes.ELEM_F32, row=100, n=3, vocab=100, t=0, k=0, p=0, m=0, u=A, ids=A, lp=0, ws=A, ws_bytes=None):
    L = oes.lib()
    if ws_bytes is None:
        b = ctypes.c_int64()
        assert L.oes_sample_workspace(3, 100, ctypes.byref(b)) == oes.OK
        ws_bytes = b.value
    return L.oes_sample(logits, elem, row, n, vocab, t, k, p, m, u, ids, lp, ws, ws_bytes, None)


def test_sample_refuses():
    for bad in (dict(logits=0), dict(logits=A + 2), dict(u=0), dict(ids=0), dict(t=A + 2), dict(k=A + 1), dict(p=A + 3),
                dict(m=A + 2), dict(u=A + 2), dict(ids=A + 2), dict(lp=A + 1), dict(row=99), dict(n=-1), dict(vocab=0),
                dict(elem=oes.ELEM_BF16, logits=A + 1), dict(ws=0), dict(ws=A + 8), dict(ws_bytes=0)):
        assert sample(**bad) == oes.ERR_ARG, bad
    for bad in (dict(elem=oes.ELEM_FP16), dict(n=(1 << 16) + 1), dict(vocab=(1 << 20) + 1, row=1 << 21)):
        assert sample(**bad) == oes.ERR_UNSUPPORTED, bad
    assert sample(n=1 << 16, vocab=1 << 20, row=1 << 20, ws_bytes=1 << 50) == oes.ERR_UNSUPPORTED   # beyond a launch
    assert sample(n=0, logits=0, u=0, ids=0, ws=0, ws_bytes=0) == oes.OK
    b = ctypes.c_int64()
    assert oes.lib().oes_sample_workspace(3, 100, None) == oes.lib().oes_sample_workspace(-1, 100, ctypes.byref(b)) == oes.ERR_ARG


# ------------------------------------------------------------------ the binding's own checks (CPU tensors end there)
def refused(call, *words):
    with pytest.raises(oes.OesError) as e:
        call()
    assert e.value.status == oes.ERR_ARG
    assert not words or any(w in str(e.value) for w in words), str(e.value)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refuses_norms():
    x, w = bf(3, 64), oes.Norm(bf(64))
    refused(lambda: oes.norm(x, bf(3, 64), pre=w), "not on a GPU")
    for call in (lambda: oes.norm(bf(64), bf(64), pre=w), lambda: oes.norm(x, bf(3, 32), pre=w),
                 lambda: oes.norm(x, torch.zeros(3, 64), pre=w), lambda: oes.norm(x.half(), bf(3, 64), pre=w),
                 lambda: oes.norm(x, bf(3, 64), pre=oes.Norm(bf(32))), lambda: oes.norm(x, bf(3, 128)[:, ::2], pre=w),
                 lambda: oes.norm(x, bf(3, 64), res=bf(3, 64), res_out=torch.zeros(3, 64)),
                 lambda: oes.norm(x, bf(3, 64), res=torch.zeros(3, 64).half()),
                 lambda: oes.norm(x, bf(3, 64), gate=bf(2, 64)), lambda: oes.norm(x, bf(3, 64), gate=torch.zeros(3, 64)),
                 lambda: oes.norm(x, bf(3, 64), gate=bf(3, 128)[:, ::2]),
                 lambda: oes.Norm(bf(64), bias=torch.zeros(64)), lambda: oes.Norm(bf(64), bias=bf(32)),
                 lambda: oes.Norm(bf(2, 32)), lambda: oes.Norm(bf(128)[::2])):
        refused(call)


def test_binding_refuses_products():
    x, w, y = bf(3, 64), bf(10, 64), bf(3, 10)
    refused(lambda: oes.linear_bf16(x, w, y), "not on a GPU")
    for call in (lambda: oes.linear_bf16(x, bf(10, 32), y), lambda: oes.linear_bf16(x, w, bf(3, 9)),
                 lambda: oes.linear_bf16(x, w, bf(2, 10)), lambda: oes.linear_bf16(x, w, y, act="swiglu"),
                 lambda: oes.linear_bf16(x.float(), w, y), lambda: oes.linear_bf16(x, w, y.half()),
                 lambda: oes.linear_bf16(x, w, y, bias=bf(9)), lambda: oes.linear_bf16(x, w, y, bias=torch.zeros(10)),
                 lambda: oes.linear_bf16(x, w, y, res=torch.zeros(3, 10)), lambda: oes.linear_bf16(x, w, y, res=bf(3, 9)),
                 lambda: oes.linear_bf16(bf(3, 128)[:, ::2], w, y), lambda: oes.linear_bf16(x[0], w, y),
                 lambda: oes.linear_bf16(x, w, bf(10, 3).t())):
        refused(call)


def test_binding_refuses_sampling():
    logits, u, ids, ws = torch.zeros(3, 50), torch.zeros(3), torch.zeros(3, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    refused(lambda: oes.sample(logits, u, ids, ws), "not on a GPU")
    for call in (lambda: oes.sample(logits[0], u, ids, ws), lambda: oes.sample(logits.half(), u, ids, ws),
                 lambda: oes.sample(logits, u[:2], ids, ws), lambda: oes.sample(logits, u.double(), ids, ws),
                 lambda: oes.sample(logits, u, ids.long(), ws), lambda: oes.sample(logits, u, ids, ws, top_k=u),
                 lambda: oes.sample(logits, u, ids, ws, temperature=ids), lambda: oes.sample(logits, u, ids, ws, top_p=u[:1]),
                 lambda: oes.sample(logits, u, ids, ws, min_p=u.double()), lambda: oes.sample(logits, u, ids, ws, logprob=u.bfloat16()),
                 lambda: oes.sample(logits.t(), u, ids, ws), lambda: oes.sample(logits, u, ids, ws[::2])):
        refused(call)

"""CPU checks of the operators around the expert step: refusals of the C ABI and of the
binding before any GPU work, the page arithmetic that the kernels share with the
host, and the rotary frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

import offloaded_expert_slot_amd as oes

A = 1 << 12  # an aligned address that is never dereferenced: refusals happen before


def kv(**over):
    c = dict(k=A, v=A, table=A, len=A, status=0, k_page=1024, k_row=128, k_head=64, v_page=1024, v_row=128, v_head=64,
             table_stride=4, elem=oes.ELEM_BF16, num_pages=9, page_size=8, kv_heads=2, head_dim=64, batch=3,
             max_pages=4, k_scale=1.0, v_scale=1.0)
    c.update(over)
    return oes.Kv(*[c[f] for f, _ in oes.Kv._fields_])


BAD_KV = [dict(elem=oes.ELEM_FP16), dict(head_dim=8), dict(head_dim=72), dict(head_dim=272), dict(kv_heads=0),
          dict(kv_heads=1025), dict(page_size=0), dict(max_pages=0), dict(batch=-1), dict(batch=(1 << 20) + 1), dict(num_pages=-1),
          dict(page_size=1 << 20, max_pages=1 << 11, table_stride=1 << 11), dict(k_scale=0.0), dict(k_scale=math.nan),
          dict(v_scale=math.inf), dict(v_scale=-1.0), dict(k_scale=0.5), dict(k=0), dict(v=0), dict(table=0), dict(len=0),
          dict(table_stride=3), dict(table=A + 2), dict(status=A + 1), dict(k_head=60), dict(k_row=-128), dict(k=A + 8),
          dict(elem=oes.ELEM_E4M3, k_head=72)]


def attn(c, q=A, q_row=256, out=2 * A, o_row=256, q_heads=4, n=5, q_start=A, scale=0.125, window=0, ws=A, ws_bytes=1 << 40,
         lse=A):
    return oes.lib().oes_attn(ctypes.byref(c) if c else None, q, q_row, 64, out, o_row, 64, lse, q_heads, n, q_start, scale,
                              window, ws, ws_bytes, None)


def weigh(c, acc=A, stride=32, lse=A):
    return oes.lib().oes_attn_weigh(ctypes.byref(c), A, 256, 64, lse, 4, 5, A, 0.125, 0, acc, stride, None)


def evict(c, acc=A, stride=32, budget=8, first=1, last=2, kept=A, new_len=A, ws=A, ws_bytes=1 << 20):
    return oes.lib().oes_kv_evict(ctypes.byref(c), acc, stride, budget, first, last, kept, new_len, ws, ws_bytes, None)


def append(c, q=A, q_out=A, qo_row=256, k=A, v=A, n=5, q_start=A, rot=64, layout=0, freq=A, mscale=1.0, pos=A):
    return oes.lib().oes_rope_append(ctypes.byref(c), q, 256, 64, q_out, qo_row, 64, 4, k, 128, 64, v, 128, 64, n, q_start,
                                     rot, layout, freq, mscale, pos, None)


@pytest.mark.parametrize("bad", BAD_KV, ids=str)
def test_cache_descriptions_are_refused_everywhere(bad):
    c = kv(**bad)
    b = ctypes.c_int64()
    for st in (attn(c), weigh(c), evict(c), append(c),
               oes.lib().oes_attn_workspace(ctypes.byref(c), 4, 5, ctypes.byref(b)),
               oes.lib().oes_kv_evict_workspace(ctypes.byref(c), 8, ctypes.byref(b))):
        assert st in (oes.ERR_ARG, oes.ERR_UNSUPPORTED)
    assert oes.lib().oes_last_error()


@pytest.mark.parametrize("bad", [dict(k_row=32), dict(k_head=0), dict(v_page=0)], ids=str)
def test_overlapping_rows_are_refused_where_the_cache_is_written(bad):
    assert evict(kv(**bad)) == append(kv(**bad)) == oes.ERR_ARG


@pytest.mark.parametrize("bad", [dict(q=0), dict(q=A + 4), dict(q_row=252), dict(out=0), dict(out=A), dict(o_row=32),
                                 dict(q_heads=3), dict(q_heads=0), dict(q_heads=258), dict(n=-1), dict(q_start=0),
                                 dict(q_start=A + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                                 dict(scale=math.inf), dict(window=-1), dict(lse=A + 2)], ids=str)
def test_attn_refuses(bad):
    assert attn(kv(), **bad) == oes.ERR_ARG
    assert attn(None) == oes.ERR_ARG


def test_attn_refuses_a_short_workspace():
    c = kv(page_size=64, max_pages=1 << 14, table_stride=1 << 14)
    b = ctypes.c_int64()
    assert oes.lib().oes_attn_workspace(ctypes.byref(c), 4, 5, ctypes.byref(b)) == oes.OK
    if b.value:
        assert attn(c, ws_bytes=b.value - 1) == oes.ERR_ARG
        assert attn(c, ws_bytes=b.value, ws=0) == oes.ERR_ARG
        assert attn(c, ws_bytes=b.value, ws=A + 4) == oes.ERR_ARG
    assert oes.lib().oes_attn_workspace(ctypes.byref(c), 4, 5, None) == oes.ERR_ARG


def test_weigh_and_evict_refuse():
    assert weigh(kv(), acc=0) == weigh(kv(), acc=A + 2) == weigh(kv(), stride=31) == weigh(kv(), lse=0) == oes.ERR_ARG
    for bad in (dict(acc=0), dict(stride=31), dict(budget=0), dict(budget=(1 << 30) + 1), dict(first=-1), dict(last=-1), dict(first=5, last=4),
                dict(first=(1 << 31) - 1, last=(1 << 31) - 1), dict(kept=0), dict(new_len=0), dict(ws=0), dict(ws=A + 8),
                dict(ws_bytes=1)):
        assert evict(kv(), **bad) == oes.ERR_ARG, bad


def test_rope_refuses():
    L = oes.lib()
    for bad in (dict(q=0), dict(q_out=0), dict(qo_row=512), dict(k=0), dict(v=A + 2), dict(n=-1), dict(q_start=0),
                dict(rot=0), dict(rot=63), dict(rot=66), dict(layout=2), dict(freq=0), dict(freq=A + 4),
                dict(mscale=math.nan), dict(pos=0), dict(pos=A + 2)):
        assert append(kv(), **bad) == oes.ERR_ARG, bad
    ok = dict(x=A, x_row=256, x_head=64, y=2 * A, y_row=256, y_head=64, n=3, heads=4, head_dim=64, rot=32, layout=1)
    for bad in (dict(x=0), dict(y=0), dict(y=A, y_row=512), dict(x=A + 8), dict(y_head=32), dict(n=-1), dict(heads=0),
                dict(heads=4097), dict(head_dim=24), dict(rot=65), dict(rot=34, head_dim=32), dict(layout=-1)):
        c = {**ok, **bad}
        assert L.oes_rope(*c.values(), A, 1.0, A, None) == oes.ERR_ARG, bad


def test_linear_refuses():
    def linear(fmt=oes.NVFP4, w0=A, w1=A, w2=A, N=10, K=64, x=A, xs=64, y=A, ys=10, n=2):
        return oes.lib().oes_linear(fmt, w0, w1, w2, N, K, x, xs, y, ys, n, None)
    for fmt in (oes.BF16, oes.FP8_BLOCK128, 9):
        assert linear(fmt=fmt) == oes.ERR_UNSUPPORTED
    for bad in (dict(w0=0), dict(w1=0), dict(w2=0), dict(fmt=oes.Q4_0), dict(N=0), dict(K=0), dict(K=48), dict(K=(1 << 20) + 32),
                dict(x=0), dict(y=0), dict(n=-1), dict(w0=A + 8), dict(w1=A + 2), dict(w2=A + 1), dict(x=A + 2), dict(xs=68),
                dict(xs=32), dict(ys=9), dict(y=A + 1)):
        assert linear(**bad) == oes.ERR_ARG, bad
    for bad in (dict(N=(1 << 23) + 1, ys=1 << 24), dict(n=(1 << 19) + 1)):
        assert linear(**bad) == oes.ERR_UNSUPPORTED, bad


def test_empty_calls_do_nothing():
    assert attn(kv(), n=0) == append(kv(), n=0) == oes.OK
    none = kv(batch=0, k=0, v=0, table=0, len=0)
    assert attn(none) == weigh(none) == evict(none) == append(none) == oes.OK
    assert oes.lib().oes_linear(oes.Q4_0, None, None, None, 10, 64, None, 64, None, 10, 0, None) == oes.OK
    assert oes.lib().oes_rope(None, 64, 64, None, 64, 64, 0, 1, 64, 64, 0, None, 1.0, None, None) == oes.OK


def test_pages_and_offsets():
    """Entries through the routine that the kernels use: every entry of small tables, pages out of
    range on both sides, entries before and behind the table, and offsets beyond 32 bits."""
    rng = np.random.default_rng(3)
    for ps in (1, 7, 16, 64):
        table = rng.permutation(9)[:8].reshape(2, 4).astype(np.int32)
        table[1, 2], table[1, 3] = 9, -1
        c = kv(page_size=ps, batch=2, k_page=ps * 128, v_page=ps * 256, v_row=256)
        k, v = ctypes.c_int64(), ctypes.c_int64()

        def entry(b, j):
            return oes.lib().oes_debug_kv_entry(ctypes.byref(c), table.ctypes.data, b, j, ctypes.byref(k), ctypes.byref(v))

        for b in range(2):
            for j in range(4 * ps):
                page = int(table[b, j // ps])
                if 0 <= page < 9:
                    assert entry(b, j) == oes.OK
                    assert (k.value, v.value) == ((page * ps + j % ps) * 128, (page * ps + j % ps) * 256)
                else:
                    assert entry(b, j) == oes.ERR_ARG
            assert entry(b, -1) == entry(b, 4 * ps) == entry(b, (1 << 31) - 1) == oes.ERR_ARG
        assert entry(2, 0) == entry(-1, 0) == oes.ERR_ARG
    big = kv(num_pages=1 << 20, page_size=64, k_page=64 * 1024, v_page=64 * 1024, k_row=1024, v_row=1024)
    table = np.full((3, 4), (1 << 20) - 1, np.int32)
    k, v = ctypes.c_int64(), ctypes.c_int64()
    assert oes.lib().oes_debug_kv_entry(ctypes.byref(big), table.ctypes.data, 2, 255, ctypes.byref(k), ctypes.byref(v)) == oes.OK
    assert k.value == ((1 << 20) - 1) * 64 * 1024 + 63 * 1024 > 1 << 32


def test_rope_freqs():
    """Frequencies against their formulas, written out apart; mscale; refusals."""
    for rot in (2, 26, 64, 128):
        f, m = oes.rope_freqs(rot, 10000.0)
        ref = np.array([10000.0 ** (-2 * i / rot) for i in range(rot // 2)])
        np.testing.assert_allclose(f, ref, rtol=1e-14)
        assert m == 1.0
        np.testing.assert_allclose(oes.rope_freqs(rot, 10000.0, "linear", 4.0)[0], ref / 4, rtol=1e-14)
        if rot > 2:
            base = 10000.0 * 4.0 ** (rot / (rot - 2))
            np.testing.assert_allclose(oes.rope_freqs(rot, 10000.0, "ntk", 4.0)[0],
                                       [base ** (-2 * i / rot) for i in range(rot // 2)], rtol=1e-13)
        y, m = oes.rope_freqs(rot, 10000.0, "yarn", 8.0, 4096)
        assert abs(m - (0.1 * math.log(8) + 1)) < 1e-6
        turns = 4096 * ref / (2 * math.pi)
        # the ends of the ramp are rounded outwards, so pairs beyond both bounds are exact
        assert np.all(y[turns >= 32] >= ref[turns >= 32] / 8) and np.all(y <= ref * (1 + 1e-14))
        assert np.all(np.diff(y) < 0)
        np.testing.assert_allclose(y[0], 1.0 if 4096 / (2 * math.pi) >= 32 else 1 / 8, rtol=1e-13)
        past = np.arange(rot // 2) > rot * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000.0)) + 1
        np.testing.assert_allclose(y[past], ref[past] / 8, rtol=1e-13)
    for bad in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=64, base=1.0),
                dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling="linear", factor=0.5),
                dict(rot_dim=64, scaling="yarn", factor=math.nan), dict(rot_dim=2, scaling="ntk", factor=2.0),
                dict(rot_dim=64, scaling="yarn", factor=2.0, trained_len=0), dict(rot_dim=64, scaling=4)):
        with pytest.raises(oes.OesError) as e:
            oes.rope_freqs(**bad)
        assert e.value.status == oes.ERR_ARG


def test_binding_refuses_mixed_up_tensors():
    """Element types, shapes and layouts that the binding turns down by itself (CPU tensors)."""
    z = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    k = z(4, 8, 2, 64, **bf)
    table, n = z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32)
    good = oes.KvPages(k, k.clone(), table, n)
    for args in ((k.half(), k.half(), table, n), (k, k[:3], table, n), (k, k.to(torch.float8_e4m3fn), table, n),
                 (k[0], k[0], table, n), (k, k, table.long(), n), (k, k, table, n[:2]), (k, k, table[0], n),
                 (k.transpose(2, 3), k.transpose(2, 3), table, n)):
        with pytest.raises(oes.OesError):
            oes.KvPages(*args)
    q, start, ws = z(5, 4, 64, **bf), z(4, dtype=torch.int32), z(1024, dtype=torch.uint8)
    lse, acc = z(5, 4), z(3, 2, 16)
    for call in (lambda: oes.attn(q.half(), q.half(), good, start, 1.0, ws),
                 lambda: oes.attn(q, q[:4].clone(), good, start, 1.0, ws),
                 lambda: oes.attn(q[..., :32], q[..., :32].clone(), good, start, 1.0, ws),
                 lambda: oes.attn(q, q.clone(), good, start[:3], 1.0, ws),
                 lambda: oes.attn(q, q.clone(), good, start, 1.0, ws, lse=lse[:4]),
                 lambda: oes.attn(q, q.clone(), good, start, 1.0, ws, lse=lse.double()),
                 lambda: oes.attn(q, q.clone(), good, start, 1.0, ws),  # on the CPU
                 lambda: oes.attn_weigh(q, lse, good, start, 1.0, acc[:2]),
                 lambda: oes.attn_weigh(q, lse, good, start, 1.0, acc.double()),
                 lambda: oes.kv_evict(good, acc, 4, z(3, 2, 5, dtype=torch.int32), n, ws),
                 lambda: oes.kv_evict(good, acc, 4, z(3, 2, 4), n, ws),
                 lambda: oes.rope(q, q[:4], z(32, dtype=torch.float64), z(5, dtype=torch.int32)),
                 lambda: oes.rope(q, q, z(32), z(5, dtype=torch.int32)),
                 lambda: oes.rope(q, q, z(32, dtype=torch.float64), z(5, dtype=torch.int64)),
                 lambda: oes.rope_append(q, q, k[:, 0], k[0], z(32, dtype=torch.float64), z(4, dtype=torch.int32), good, start),
                 lambda: oes.linear("q4_0", z(2, 64, **bf), [z(10, 32, dtype=torch.uint8), z(10, 2)], z(2, 10, **bf)),
                 lambda: oes.linear("q4_0", z(2, 64, **bf), [z(10, 31, dtype=torch.uint8), z(10, 2).half()], z(2, 10, **bf)),
                 lambda: oes.linear("q4_0", z(2, 64), [z(10, 32, dtype=torch.uint8), z(10, 2).half()], z(2, 10, **bf)),
                 lambda: oes.linear("nvfp4", z(2, 64, **bf), [z(10, 32, dtype=torch.uint8)], z(2, 10, **bf)),
                 lambda: oes.linear("q4_0", z(64, 2, **bf).t(), [z(10, 32, dtype=torch.uint8), z(10, 2).half()],
                                    z(2, 10, **bf))):
        with pytest.raises(oes.OesError) as e:
            call()
        assert e.value.status == oes.ERR_ARG

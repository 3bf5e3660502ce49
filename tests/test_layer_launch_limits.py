"""Calls whose launches would pass a GPU launch's 2^31 - 1 workgroups or 2^32 - 1 work-items are refused before the
first of them, by the call and by its workspace query (host code; nothing is launched)."""
import ctypes

import pytest

import offloaded_expert_slot_amd as oes

A = 1 << 12  # an aligned address that is never dereferenced


def kv(**over):
    c = dict(k=A, v=A, table=A, len=A, status=0, k_page=1024, k_row=128, k_head=128, v_page=1024, v_row=128, v_head=128,
             table_stride=4, elem=oes.ELEM_BF16, num_pages=9, page_size=8, kv_heads=1, head_dim=128, batch=1,
             max_pages=4, k_scale=1.0, v_scale=1.0)
    c.update(over)
    return oes.Kv(*[c[f] for f, _ in oes.Kv._fields_])


def evict(c):
    return oes.lib().oes_kv_evict(ctypes.byref(c), A, 64, 8, 1, 2, A, A, A, 1 << 40, None)


def evict_workspace(c):
    b = ctypes.c_int64()
    return oes.lib().oes_kv_evict_workspace(ctypes.byref(c), 8, ctypes.byref(b))


# batch * kv_heads * columns workgroups of 1024: a column is 128 bytes of a k or v row
EVICT = [(oes.ELEM_BF16, 128, 4), (oes.ELEM_BF16, 64, 2), (oes.ELEM_BF16, 80, 4), (oes.ELEM_BF16, 256, 8), (oes.ELEM_E4M3, 128, 2),
         (oes.ELEM_E4M3, 16, 2), (oes.ELEM_E4M3, 144, 4)]


@pytest.mark.parametrize("elem,D,columns", EVICT)
def test_evictions_beyond_a_launch_are_refused_whole(elem, D, columns):
    heads = 16
    most = ((1 << 22) - 1) // (heads * columns)   # sequences: their workgroups of 1024 stay below 2^32 work-items
    d = dict(elem=elem, head_dim=D, kv_heads=heads, k_head=256, v_head=256, k_row=4096, v_row=4096, k_page=1 << 16, v_page=1 << 16)
    assert evict_workspace(kv(batch=most, **d)) == oes.OK
    for batch in (most + 1, 1 << 20):
        assert evict_workspace(kv(batch=batch, **d)) == oes.ERR_UNSUPPORTED, batch
        assert evict(kv(batch=batch, **d)) == oes.ERR_UNSUPPORTED, batch
        assert b"launch" in oes.lib().oes_last_error()


def test_the_largest_batch_of_single_heads():
    assert evict(kv(batch=1 << 20)) == evict_workspace(kv(batch=1 << 20)) == oes.ERR_UNSUPPORTED
    assert evict_workspace(kv(batch=(1 << 20) - 1)) == oes.OK


def attn(c, q_heads, n):
    return oes.lib().oes_attn(ctypes.byref(c), A, 1024, 128, 2 * A, 1024, 128, None, q_heads, n, A, 0.125, 0, A, 1 << 45, None)


def attn_workspace(c, q_heads, n):
    b = ctypes.c_int64()
    return oes.lib().oes_attn_workspace(ctypes.byref(c), q_heads, n, ctypes.byref(b))


def test_attention_beyond_a_launch_is_refused_whole():
    # decode steps: a joining workgroup of 256 for each (row, head) of rows that several workgroups may share
    long = dict(batch=1 << 18, kv_heads=64, k_head=128, v_head=128, k_row=8192, v_row=8192, k_page=1 << 16, v_page=1 << 16, page_size=64,
                max_pages=64, table_stride=64)
    for n in (1 << 18, (1 << 18) - 1):
        want = oes.ERR_UNSUPPORTED if n * 64 >= 1 << 24 else oes.OK
        assert attn_workspace(kv(**long), 64, n) == want, n
    assert attn(kv(**long), 64, 1 << 18) == oes.ERR_UNSUPPORTED
    # prompts: workgroups of 256 for each (tile of rows, cache head)
    short = {**long, "batch": 1, "kv_heads": 1024, "k_row": 1 << 17, "v_row": 1 << 17, "k_page": 1 << 20, "v_page": 1 << 20}
    n = 128 << 14                                 # 2^14 tiles of 128 rows, 2^10 heads: 2^24 workgroups
    assert attn_workspace(kv(**short), 1024, n) == attn(kv(**short), 1024, n) == oes.ERR_UNSUPPORTED
    assert attn_workspace(kv(**short), 1024, n - 128) == oes.OK


def test_entry_weights_beyond_a_launch_are_refused():
    # prompts: a workgroup of 512 for each 128 entries of the table's width, cache head and sequence
    c = kv(batch=1, kv_heads=1, page_size=1 << 10, max_pages=1 << 20, table_stride=1 << 20)
    assert c.page_size * c.max_pages == 1 << 30
    c.kv_heads, c.k_head, c.v_head = 2, 128, 128
    c.batch = 1
    # 2^23 workgroups of 128 entries a head: 2 heads make 2^24 of 512 = 2^33 work-items
    assert oes.lib().oes_attn_weigh(ctypes.byref(c), A, 1024, 128, A, 2, 100, A, 0.125, 0, A, 1 << 30, None) == oes.ERR_UNSUPPORTED
    c.max_pages = c.table_stride = 1 << 19        # 2^22 * 2 of 512: 2^32
    assert oes.lib().oes_attn_weigh(ctypes.byref(c), A, 1024, 128, A, 2, 100, A, 0.125, 0, A, 1 << 30, None) == oes.ERR_UNSUPPORTED


def test_more_rows_than_the_kernels_count_are_refused():
    """Row numbers stay below 2^30, so that a sum of two of them stays within 32 bits."""
    c = kv()
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert attn(c, 1, n) == attn_workspace(c, 1, n) == oes.ERR_UNSUPPORTED, n
        assert oes.lib().oes_attn_weigh(ctypes.byref(c), A, 1024, 128, A, 1, n, A, 0.125, 0, A, 32, None) == oes.ERR_UNSUPPORTED, n

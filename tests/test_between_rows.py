"""Rows that a norm writes may lie in any order and distance, but share no element (CPU: checks before any launch)."""
import ctypes
import random

import offloaded_expert_slot_amd as oes

A = 1 << 12  # an aligned address that is never dereferenced


def norm(written, n, heads, dim, row, head):
    """Status of a call whose rows of `written` lie so: refused for a last argument where they do not overlap."""
    spec = oes.NormSpec(0, 0, 0, oes.ELEM_BF16, 1e-6, 0.0)
    c = dict(post=0, pre=ctypes.addressof(spec), x=A, gate=A + 1, res=2 * A, res_out=3 * A, y=4 * A, x_row=0, x_head=0, gate_row=0,
             gate_head=0, gate_col=0, res_row=0, res_head=0, ro_row=heads * dim, ro_head=dim, y_row=heads * dim, y_head=dim, n=n,
             heads=heads, dim=dim, x_elem=oes.ELEM_BF16, res_elem=oes.ELEM_BF16, gate_act=0, scale=1.0, reserved=0)
    c.update({"y": dict(y_row=row, y_head=head), "res_out": dict(ro_row=row, ro_head=head)}[written])
    args = oes.NormArgs(*[c[f] for f, _ in oes.NormArgs._fields_])
    assert oes.lib().oes_norm(ctypes.byref(args), None) == oes.ERR_ARG   # the gate's address is odd: nothing runs
    return oes.lib().oes_last_error().decode()


def refused(*args):
    error = norm(*args)
    assert ("overlap" in error) != ("gate" in error), error
    return "overlap" in error


def test_rows_that_overlap_are_refused():
    for written in ("y", "res_out"):
        assert refused(written, 5, 2, 64, 64, 64)          # token 0's head 1 is token 1's head 0
        assert refused(written, 5, 2, 64, 120, 64)
        assert refused(written, 5, 2, 64, 64, 312)
        assert refused(written, 2, 5, 64, 64, 64)
        assert refused(written, 2, 2, 64, 0, 64) and refused(written, 2, 2, 64, 64, 0)
        assert refused(written, 40000, 50000, 8, 8 * 50000 - 8, 8)
        assert not refused(written, 5, 2, 64, 128, 64)
        assert not refused(written, 5, 2, 64, 64, 320)     # heads before tokens
        assert not refused(written, 5, 2, 64, 1 << 40, 1 << 20)
        assert not refused(written, 5, 2, 64, 1 << 20, 1 << 62)
        assert not refused(written, 40000, 50000, 8, 8 * 50000, 8)
        assert not refused(written, 40000, 50000, 8, 8, 8 * 40000)
        assert not refused(written, 2, 2, 64, 192, 128)    # 0, 128, 192, 320: in turns
        assert not refused(written, 7, 1, 64, 64, 0) and not refused(written, 1, 7, 64, 0, 64)


def test_random_rows():
    rng = random.Random(3)
    seen = set()
    for _ in range(4000):
        n, heads, dim = rng.randint(1, 6), rng.randint(1, 6), 8 * rng.randint(1, 4)
        row, head = 8 * rng.randint(0, 40), 8 * rng.randint(0, 40)
        starts = sorted(t * row + h * head for t in range(n) for h in range(heads))
        want = any(b - a < dim for a, b in zip(starts, starts[1:]))
        assert refused(rng.choice(["y", "res_out"]), n, heads, dim, row, head) == want, (n, heads, dim, row, head)
        seen.add(want)
    assert len(seen) == 2

"""Every shape of the bf16 product's tiles is run by a GPU test, with its main loop (CPU: the rule alone)."""
import math
import random

from tests import product_shapes as S


def test_cases_reach_every_shape_and_its_main_loop():
    shapes = S.table()
    seen = {}
    for n, N, K, act in S.CASES:
        i, once, trips, part = S.picked(shapes, n, N, K, act)
        assert trips >= 2 and part, (n, N, K, act, i, trips)
        seen.setdefault((i, act == "swiglu", once), []).append((n, N, K))
    for i, (BM, BN, _, _, _) in enumerate(shapes):
        for swiglu in (False, True):
            got = [c for c in seen if c[:2] == (i, swiglu)]
            assert got, (i, swiglu)
            # some whose rows, and some whose tokens, end inside a tile
            sizes = [s for c in got for s in seen[c]]
            assert any(n % BM for n, _, _ in sizes) and any(N * (1 + swiglu) % BN for _, N, _ in sizes), (i, swiglu)
    # no call takes a kernel that the cases do not
    rng = random.Random(11)
    for _ in range(40000):
        n, N = (int(math.exp(rng.uniform(math.log(a), math.log(b)))) for a, b in ((2, 1 << 16), (1, 1 << 20)))
        act = rng.choice(["none", "swiglu"])
        i, once, _, _ = S.picked(shapes, n, N, 64, act)
        assert (i, act == "swiglu", once) in seen, (n, N, act, i, once)

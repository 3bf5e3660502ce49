"""The rule by which the bf16 product takes a shape, read from the kernel's source and evaluated here (not a test module),
and sizes that reach every shape's main loop."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "offloaded_expert_slot_amd", "csrc",
                      "k_linear_bf16.hip")


def table():
    """[(BM, BN, WK, S, cost)] of the shapes in order."""
    text = open(SOURCE).read()
    cost = [int(c) for c in re.search(r"const int cost\[\] = \{([^}]*)\}", text).group(1).split(",")]
    shapes = re.findall(r"typedef Shape<([^>]*)> P(\d+);", text)
    assert [int(i) for _, i in shapes] == list(range(len(cost)))
    rows = [[int(v) for v in s.split(",")] for s, _ in shapes]
    return [(r[0], r[1], r[4], r[5], c) for r, c in zip(rows, cost)]


def picked(shapes, n, N, K, act):
    """(shape's number, whether one tile of tokens reads W, trips of the main loop of the group of waves with the fewest
    steps, whether the last step is a part) of a call of n > 1 tokens."""
    rows = N * (2 if act == "swiglu" else 1)

    def tiles(s):
        return -(-rows // s[1]) * -(-n // s[0])

    best = min(range(len(shapes)), key=lambda i: (-(-tiles(shapes[i]) // 256) * shapes[i][4], i))
    BM, _, WK, S, _ = shapes[best]
    whole = (K + 63) // 64 // WK
    trips = max(0, -(-(whole - 2 * S) // S))
    return best, BM <= 64 and n <= BM, trips, K % 64 != 0


# (n, N, K, act): every shape with and without SwiGLU, and where it can be with one tile of tokens and with several; two
# trips or more of the main loop, a last step in part, and rows and tokens that end inside a tile
CASES = [
    # 16 x 16
    (13, 9, 5320, "none"), (17, 9, 5320, "none"), (5, 1001, 5320, "none"), (15, 9, 5320, "swiglu"),
    (70, 25, 5320, "swiglu"),
    # 16 x 32
    (2, 4097, 2632, "none"), (16, 8003, 4104, "none"), (17, 2049, 2632, "none"), (9, 2050, 2632, "swiglu"),
    (24, 2045, 7176, "swiglu"), (17, 1041, 2632, "swiglu"),
    # 32 x 16
    (96, 1350, 2888, "none"), (4104, 9, 2632, "none"), (2075, 17, 2632, "swiglu"), (96, 675, 2888, "swiglu"),
    # 32 x 32
    (17, 4100, 2632, "none"), (600, 411, 2632, "none"), (31, 2049, 2632, "swiglu"), (4102, 9, 2664, "swiglu"),
    # 64 x 32
    (33, 4134, 2648, "none"), (514, 515, 2648, "none"), (63, 2049, 2632, "swiglu"), (4150, 17, 2632, "swiglu"),
    # 64 x 64
    (17, 8226, 1288, "none"), (65, 4138, 1304, "none"), (50, 4185, 1288, "swiglu"), (65, 2058, 1288, "swiglu"),
    # 64 x 128
    (2, 24811, 840, "none"), (333, 2877, 2888, "none"), (2, 12405, 840, "swiglu"), (65, 4105, 840, "swiglu"),
    (1030, 1667, 904, "none"),
    # 128 x 128
    (130, 10921, 648, "none"), (65, 8229, 664, "swiglu"), (2100, 7169, 1032, "none"),
    # 256 x 128
    (260, 13186, 648, "none"), (1925, 2049, 712, "none"), (130, 10940, 648, "swiglu"),
    # 256 x 256
    (515, 13342, 456, "none"), (2819, 2839, 1032, "none"), (259, 11087, 456, "swiglu"), (3001, 2055, 520, "swiglu"),
]

"""Products for each kernel: (way, rows of each group, N, K). Of the rows LEAD before the first group and
TAIL after the last belong to none. test_matmul_rule_cpu.py holds the rule to the kernels named here."""
LEAD, TAIL = 3, 5

GROUPED = {
    "stream": [
        ("fwd", (4, 0, 9, 1, 0, 2, 0, 0), 264, 1032),     # four rows of x at a time
        ("fwd", (5, 2), 136, 2056),                       # sixteen
        ("fwd", (1, 0, 30), 72, 520),                     # a small output
    ],
    "split32": [
        ("fwd", (100, 0, 1, 31, 33), 520, 1032), ("dx", (1, 0, 32, 7), 1096, 136), ("dx", (33, 64), 520, 264),
        ("dw", (1, 2200, 0, 63), 136, 40), ("dw", (1300,), 72, 264),
    ],
    "tile64_parts": [
        ("fwd", (70, 0, 17), 4104, 840), ("dx", (17, 0, 33, 1), 1032, 3080), ("dw", (800, 0, 2400, 1), 264, 520),
    ],
    "tile64": [
        ("fwd", (200, 0, 65, 1), 2056, 264), ("dx", (64, 0, 129), 72, 3992), ("dw", (1, 0, 90, 200), 712, 520),
    ],
    "tile128_deep": [
        ("fwd", (129, 0, 383), 4104, 584), ("dx", (600, 1), 1096, 4104), ("dw", (1, 0, 1600), 1032, 904),
    ],
    "tile128": [
        ("fwd", (1, 0, 128, 130, 900), 4104, 72), ("dx", (700, 0, 257), 264, 4104), ("dw", (1, 0, 200, 129), 2056, 1096),
    ],
    "tile256": [
        # ragged and empty groups, row tiles of 1 and of 128 rows and less, tiles cut in two
        ("fwd", (1, 129, 0, 1962), 2904, 2904), ("dx", (1, 129, 0, 1962), 2904, 2904), ("dw", (1, 129, 0, 1962), 2904, 2904),
        # many groups of few tiles; a last step of 8 values; columns that end inside a half
        ("fwd", (256, 128, 257, 700, 0, 384, 512, 1), 2056, 1032), ("dx", (256, 128, 257, 700, 0, 384, 512, 1), 1032, 2056),
        # one to several steps, the last whole and not, of one group and the next
        ("dw", (1, 64, 65, 0, 128, 2900), 1496, 1032),
        # several tiles a block
        ("fwd", (3100, 3400), 4360, 520), ("dx", (3100, 3400), 520, 4360), ("dw", (700, 0, 900, 600), 3848, 2904),
        ("fwd", (4592,), 4616, 512), ("dx", (4592,), 512, 4616),
    ],
}

# (T, N, K) of linear
LINEAR = {
    "stream": [(3, 264, 1032), (15, 136, 2056)],
    "split32": [(100, 520, 1032)],
    "tile64_parts": [(70, 5000, 840)],
    "tile64": [(300, 2056, 264)],
    "tile128_deep": [(500, 5000, 584)],
    "tile128": [(1100, 4104, 72)],
    "tile256": [(2100, 2904, 2904), (4600, 4616, 520)],
}

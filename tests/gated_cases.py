"""Gated blocks for each product kernel: (kernel, rows of each group, h, d). Of the rows LEAD before the first
group and TAIL after the last belong to none. test_gated_cpu.py holds the rule to the kernels named here."""
LEAD, TAIL = 3, 5

FORWARD = [
    ("stream", (4, 0, 9, 1, 0, 2, 0, 0), 136, 1032),   # four rows of x at a time
    ("stream", (5, 2), 72, 2056),                      # sixteen
    ("stream", (1,), 8, 8),
    ("split32", (100, 0, 1, 31, 33), 264, 1032),
    ("tile64_parts", (70, 0, 17), 2056, 840),
    ("tile64", (200, 0, 65, 1), 1032, 264),
    ("tile128_deep", (129, 0, 383), 2056, 584),
    ("tile128", (1, 0, 128, 130, 900), 2056, 72),
    ("tile256", (1, 129, 0, 1962), 1448, 2904),
    ("tile256", (256, 128, 257, 700, 0, 384, 512, 1), 1032, 1032),
    ("tile256", (4592,), 2312, 512),
]

BACKWARD = [
    ("split32", (1, 0, 32, 7), 136, 1096),
    ("split32", (33, 64), 264, 520),
    ("tile64_parts", (17, 0, 33, 1), 3080, 1032),
    ("tile64", (64, 0, 129), 3992, 72),
    ("tile64", (1,), 8, 8),
    ("tile128_deep", (600, 1), 4104, 1096),
    ("tile128", (700, 0, 257), 4104, 264),
    ("tile256", (1, 129, 0, 1962), 2904, 2904),
    ("tile256", (256, 128, 257, 700, 0, 384, 512, 1), 2056, 1032),
    ("tile256", (4592,), 4616, 512),
]

# (kernel, T, h, d) of one dense block
DENSE = [("stream", 1, 264, 1032), ("stream", 13, 136, 2056), ("split32", 100, 264, 1032), ("tile64_parts", 70, 2504, 840),
         ("tile64", 300, 1032, 264), ("tile128_deep", 500, 2504, 584), ("tile128", 1100, 2056, 72), ("tile256", 2100, 1448, 2904)]

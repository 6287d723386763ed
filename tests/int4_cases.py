"""Products with 4-bit weights for each shape of the kernel: (shape, rows of each group, N, K) and (shape, T, N, K) of a dense
one. Of the rows LEAD before the first group and TAIL after the last belong to none."""
LEAD, TAIL = 3, 5

GROUPED = [
    ("few_wide", (4, 0, 9, 1, 0, 2, 0, 0), 272, 1152), ("few", (4, 0, 9, 1, 0, 2, 0, 0), 2064, 640),
    ("rows16", (5, 0, 17, 2), 144, 2176), ("rows32", (33, 0, 40, 1), 208, 384), ("rows64", (129, 0, 1, 63), 336, 896),
    ("tile64", (200, 0, 65, 1), 656, 512), ("tile128", (1, 700, 129, 2000), 1296, 1152),
]
DENSE = [
    ("few_wide", 1, 16, 128), ("few_wide", 1, 144, 5120), ("few_wide", 4, 272, 1152), ("few", 3, 16400, 384), ("rows16", 5, 80, 1280),
    ("rows16", 16, 1040, 256), ("rows32", 17, 208, 2176), ("rows32", 32, 64, 128), ("rows64", 37, 336, 1152), ("rows64", 64, 128, 256),
    ("tile64", 65, 144, 1280), ("tile64", 511, 400, 128), ("tile128", 513, 528, 640), ("tile128", 1100, 272, 384),
]

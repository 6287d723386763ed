"""The rule that picks a product's kernel (csrc/matmul_rule.h), asked through a small host program."""
import os
import subprocess

import pytest

import matmul_cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_ffn_int4_amd", "csrc")
MODES = {"fwd": 0, "dx": 1, "dw": 2}


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rule") / "rule")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "matmul_rule_main.cpp")], check=True)

    def ask(*cases):
        lines = "".join("%d %d %d %d %d\n" % (MODES[way], P, E, N, K) for way, P, E, N, K in cases)
        return subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.split()

    return ask


@pytest.mark.parametrize("way,P,E,N,K,kernel", [
    # groups shorter than a tile have one whole tile each: 48 rows over 128 experts are about 40
    # row tiles of 32 (x 8 columns = 320), 15 over 2 two (x 152 = 304), 42 over 16 fifteen (x 21),
    # 12 over 4 four (x 105)
    ("dx", 48, 128, 8896, 232, "tile64_parts"),
    ("dx", 15, 2, 5360, 4840, "tile64_parts"),
    ("dx", 42, 16, 4880, 664, "tile64_parts"),
    ("dx", 12, 4, 11928, 3336, "tile64_parts"),
    # 5 rows in each of 128: 128 row tiles of 64, x 3 columns
    ("dx", 640, 128, 1024, 136, "tile64"),
    # groups longer than a tile count as before: their last tile is half empty
    ("dx", 640, 4, 1024, 136, "split32"),
    ("dx", 3, 1, 8704, 136, "split32"),
    ("dx", 300, 16, 512, 1024, "tile64"),
])
def test_groups_shorter_than_a_tile(rule, way, P, E, N, K, kernel):
    assert rule((way, P, E, N, K)) == [kernel]


def test_cases_of_each_kernel(rule):
    """What the GPU tests call a kernel's sizes are the sizes that the rule sends to it."""
    for kernel, cases in matmul_cases.GROUPED.items():
        for way, counts, N, K in cases:
            P = sum(counts) + matmul_cases.LEAD + matmul_cases.TAIL
            assert rule((way, P, len(counts), N, K)) == [kernel], (way, counts, N, K)
    for kernel, cases in matmul_cases.LINEAR.items():
        for T, N, K in cases:
            assert rule(("fwd", T, 1, N, K)) == [kernel], (T, N, K)

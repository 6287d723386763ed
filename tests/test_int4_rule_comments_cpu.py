"""The products that the table of 4-bit shapes names beside each shape are sent to that shape."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RULE = os.path.join(ROOT, "moe_ffn_int4_amd", "csrc", "int4_rule.h")
PRODUCT = re.compile(r"(\d+) (?:over E = (\d+), |x )(\d+) x (\d+) (\d+(?:\.\d+)?)")


def _named():
    """(shape, P, E, N, K) of the comments in the table of costs."""
    with open(RULE) as f:
        text = f.read()
    shapes = re.findall(r"^    k(\d+x\d+(?:p\d+)?),$", text, re.M)
    rows = text[text.index("kInt4Costs[] = {"):].split("\n")[1:]
    named, pending = [], []
    for line in rows:
        line = line.strip()
        if line.startswith("//"):
            pending += [(int(p), int(e or 1), int(n), int(k)) for p, e, n, k, _ in PRODUCT.findall(line)]
        elif line.startswith("{"):
            named.append((shapes[len(named)], pending))
            pending = []
        else:
            break
    assert [s for s, _ in named] == shapes
    return named


def test_each_shape_has_a_product_that_it_is_chosen_for(tmp_path):
    named = _named()
    assert all(products for _, products in named), [s for s, p in named if not p]
    exe = str(tmp_path / "rule")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.dirname(RULE), "-o", exe, os.path.join(ROOT, "tests", "int4_rule_main.cpp")], check=True)
    want = [(shape, p) for shape, products in named for p in products]
    got = subprocess.run([exe], input="\n".join("%d %d %d %d 128" % p for _, p in want), capture_output=True, text=True, check=True).stdout.split()
    wrong = [f"{p}: named at {shape}, sent to {g}" for (shape, p), g in zip(want, got) if g != shape]
    assert not wrong, wrong


@pytest.mark.parametrize("text,found", [("// 59 x 2800 x 256 3.6 (k32x64p4 3.9)", [("59", "", "2800", "256", "3.6")]),
                                        ("// 10 over E = 16, 5248 x 1664 11.6 (k16x256 14.0)", [("10", "16", "5248", "1664", "11.6")])])
def test_how_comments_are_read(text, found):
    assert PRODUCT.findall(text) == found

"""Refusals of the products with 4-bit weights, before any HIP call; the shapes that the rule picks; their LDS on every device."""
import os
import subprocess

import pytest

import moe_ffn_int4_amd as moe
from int4_cases import DENSE, GROUPED, LEAD, TAIL
from test_lds_limit_cpu import _run

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID = 0, 1
F = 0x10000000000  # aligned addresses, far apart, never dereferenced


def at(i):
    return F + i * (1 << 44)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from moe_ffn_int4_amd import build
        build.build()
    return moe.lib()


GROUPS = dict(x=at(0), q=at(1), scales=at(2), off=at(3), P=64, E=4, N=128, K=256, group=128, y=at(4), fp32=0)
LINEAR = dict(x=at(0), q=at(1), scales=at(2), bias=at(3), act=2, residual=at(4), T=64, N=128, K=256, group=128, y=at(5), fp32=0)


def call(L, which, **kw):
    v = {**(GROUPS if which == "grouped" else LINEAR), **kw}
    assert len(v) == (11 if which == "grouped" else 12)
    return (L.moe_grouped_matmul_int4 if which == "grouped" else L.moe_linear_int4)(*v.values(), None)


BOTH = [(dict(N=0), "N = 0"), (dict(N=8), "N = 8"), (dict(N=24), "N = 24"), (dict(N=(1 << 20) + 16), "N ="), (dict(K=64), "K = 64"), (dict(K=0), "K = 0"),
        (dict(K=200), "K = 200"), (dict(K=(1 << 20) + 128), "K ="), (dict(group=16), "group_size 16"), (dict(group=0), "group_size 0"),
        (dict(group=256), "group_size 256"), (dict(x=None), "x is NULL"), (dict(q=None), "q is NULL"), (dict(scales=None), "scales is NULL"),
        (dict(y=None), "y is NULL"), (dict(x=at(0) + 2), "aligned"), (dict(q=at(1) + 8), "aligned"), (dict(scales=at(2) + 4), "aligned"),
        (dict(y=at(0) + 64), "y overlaps x"), (dict(y=at(1)), "y overlaps q"), (dict(y=at(2)), "y overlaps scales"),
        (dict(group=32, y=at(2) + 128 * 8 * 4 - 16), "y overlaps scales")]


@pytest.mark.parametrize("which,kw,needle", [("grouped", *c) for c in BOTH] + [("linear", *c) for c in BOTH] + [
    ("grouped", dict(P=-1), "P = -1"), ("grouped", dict(P=(1 << 30) + 1), "P ="), ("grouped", dict(E=0), "E = 0"), ("grouped", dict(E=257), "E = 257"),
    ("grouped", dict(off=None), "offsets is NULL"), ("grouped", dict(off=at(3) + 2), "offsets"), ("grouped", dict(y=at(3)), "y overlaps offsets"),
    ("grouped", dict(E=256, N=1 << 18, K=1 << 16), "1 TiB"), ("grouped", dict(P=1 << 29, N=4096), "too many tiles"),
    ("linear", dict(T=-1), "P = -1"), ("linear", dict(act=5), "act 5"), ("linear", dict(act=-1), "act -1"), ("linear", dict(bias=at(3) + 4), "bias"),
    ("linear", dict(residual=at(4) + 2), "residual"), ("linear", dict(y=at(3)), "y overlaps bias"), ("linear", dict(y=at(4) + 16), "y overlaps residual"),
    ("linear", dict(y=at(4), fp32=1), "y overlaps residual"),
])
def test_refusals(L, which, kw, needle):
    assert call(L, which, **kw) == INVALID
    said = L.moe_last_error().decode()
    assert needle in said, said


def test_calls_that_are_allowed(L):
    """They end at the device here, past the checks."""
    assert call(L, "grouped", P=0, x=None, q=None, y=None) == OK and call(L, "linear", T=0, x=None, y=None) == OK
    for which, kw in (("grouped", {}), ("grouped", dict(E=1, off=None)), ("linear", dict(bias=None, residual=None, act=0)), ("linear", dict(y=at(4)))):
        assert call(L, which, **kw) != INVALID, L.moe_last_error()


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("rule") / "rule")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "moe_ffn_int4_amd", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "int4_rule_main.cpp")], check=True)
    return exe


def test_the_cases_reach_every_shape(rule):
    lines, want = [], []
    for shape, counts, N, K in GROUPED:
        lines.append(f"{sum(counts) + LEAD + TAIL} {len(counts)} {N} {K} 128")
        want.append(shape)
    for shape, T, N, K in DENSE:
        lines.append(f"{T} 1 {N} {K} 128")
        want.append(shape)
    got = subprocess.run([rule], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    assert got == want
    assert set(got[:len(GROUPED)]) == set(got[len(GROUPED):]) == set(subprocess.run([rule, "names"], capture_output=True, text=True).stdout.split())


CHILD = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
L.moe_grouped_matmul_int4.argtypes = [P, P, P, P, i64, i64, i64, i64, i32, P, i32, P]
L.moe_linear_int4.argtypes = [P, P, P, P, i32, P, i64, i64, i64, i32, P, i32, P]
L.moe_last_error.restype = ctypes.c_char_p
at = [0x10000000000 + i * (1 << 44) for i in range(5)]  # aligned addresses, far apart, never read
for device in (0, 1, 63, 0):
    stub.stub_set_device(device)
    for line in sys.argv[3:]:
        way, p, e, n, k = line.split(",")
        p, e, n, k = int(p), int(e), int(n), int(k)
        for group in (128, 64, 32):
            if way == "grouped":
                st = L.moe_grouped_matmul_int4(at[0], at[1], at[2], at[3], p, e, n, k, group, at[4], 0, None)
            else:
                st = L.moe_linear_int4(at[0], at[1], at[2], None, 0, None, p, n, k, group, at[4], 0, None)
            assert st == 0, (line, st, L.moe_last_error())
out = (ctypes.c_int * 3)()
stub.stub_counts(out)
print(*out)
"""


def test_lds_of_every_shape_on_every_device(L, tmp_path):
    lines = [f"grouped,{sum(c) + LEAD + TAIL},{len(c)},{n},{k}" for _, c, n, k in GROUPED] + [f"linear,{t},1,{n},{k}" for _, t, n, k in DENSE]
    launches, large, refused = _run(tmp_path, CHILD, *lines)
    assert launches == 4 * 3 * len(lines) and large > 0 and refused == 0, (launches, large, refused)

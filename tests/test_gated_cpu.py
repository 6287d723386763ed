"""Refusals of the gated block, before any HIP call; the kernels that its sizes take; their LDS on several devices."""
import os
import subprocess

import pytest

import moe_ffn_int4_amd as moe
from gated_cases import BACKWARD, DENSE, FORWARD, LEAD, TAIL
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


FWD = dict(x=at(0), w=at(1), bias=None, off=at(2), act=2, P=64, E=4, h=128, d=64, y=at(3), z=at(4))
DZ = dict(dy=at(0), w2=at(1), z=at(2), off=at(3), act=2, P=64, E=4, h=128, d=64, dz=at(4), y=at(5))


def call(L, which, **kw):
    v = {**(FWD if which == "fwd" else DZ), **kw}
    assert len(v) == 11
    return (L.moe_gated if which == "fwd" else L.moe_gated_dz)(*v.values(), None)


BOTH = [(dict(P=-1), "P = -1"), (dict(P=(1 << 30) + 1), "P ="), (dict(E=0), "E = 0"), (dict(E=257), "E = 257"), (dict(h=0), "h = 0"),
        (dict(h=12), "h = 12"), (dict(h=(1 << 19) + 8), "h ="), (dict(d=4), "d = 4"), (dict(d=(1 << 20) + 8), "d ="), (dict(act=-1), "act"),
        (dict(act=5), "act"), (dict(off=None), "offsets is NULL")]


@pytest.mark.parametrize("which,kw,needle", [("fwd", *c) for c in BOTH] + [("dz", *c) for c in BOTH] + [
    ("fwd", dict(E=256, h=8192, d=253952), "1 TiB"), ("dz", dict(E=256, h=8192, d=(1 << 18) + 8), "1 TiB"),
    ("fwd", dict(off=at(2) + 2), "offsets"), ("dz", dict(off=at(3) + 2), "offsets"),
    ("fwd", dict(h=1 << 19, d=4096), "2^31"), ("fwd", dict(h=32768 - 256 + 8, d=65536), "2^31"),
    ("fwd", dict(bias=at(6)), "bias with offsets"), ("fwd", dict(E=1, off=None, bias=at(6) + 4), "bias"),
    ("fwd", dict(x=None), "x is NULL"), ("fwd", dict(w=None), "w is NULL"), ("fwd", dict(y=None), "y is NULL"),
    ("fwd", dict(x=at(0) + 8), "aligned"), ("fwd", dict(z=at(4) + 8), "aligned"), ("fwd", dict(y=at(0) + 16), "y overlaps x"),
    ("fwd", dict(y=at(1) + 16), "y overlaps w"), ("fwd", dict(z=at(0)), "z overlaps x"), ("fwd", dict(z=at(1) + 4 * 4 * 128 * 64 - 16), "z overlaps w"),
    ("fwd", dict(z=at(3) + 64 * 128 * 2 - 16), "y overlaps z"), ("fwd", dict(y=at(2)), "y overlaps offsets"),
    ("fwd", dict(E=1, off=None, bias=at(6), y=at(6) + 1008), "y overlaps bias"),
    ("dz", dict(dy=None), "dy is NULL"), ("dz", dict(w2=None), "w2 is NULL"), ("dz", dict(z=None), "z is NULL"), ("dz", dict(dz=None), "dz is NULL"),
    ("dz", dict(z=at(2) + 2), "aligned"), ("dz", dict(y=at(5) + 8), "aligned"), ("dz", dict(dz=at(0)), "dz overlaps dy"),
    ("dz", dict(dz=at(1)), "dz overlaps w2"), ("dz", dict(dz=at(2) + 16), "dz overlaps z"), ("dz", dict(y=at(2)), "y overlaps z"),
    ("dz", dict(y=at(4) + 32), "dz overlaps y"), ("dz", dict(y=at(3)), "y overlaps offsets"),
])
def test_refusals(L, which, kw, needle):
    assert call(L, which, **kw) == INVALID
    said = L.moe_last_error().decode()
    assert needle in said, said


def test_calls_that_are_allowed(L):
    """They end at the device here, past the checks."""
    assert call(L, "fwd", P=0, x=None, y=None) == OK and call(L, "dz", P=0, dy=None, z=None) == OK
    for which, kw in (("fwd", dict(z=None)), ("fwd", dict(E=1, off=None, bias=at(6))), ("dz", dict(y=None)), ("dz", dict(dz=at(2))),
                      ("fwd", dict(h=32768 - 256, d=65536))):
        assert call(L, which, **kw) != INVALID, L.moe_last_error()


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("rule") / "rule")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "moe_ffn_int4_amd", "csrc"),
                    os.path.join(ROOT, "tests", "matmul_rule_main.cpp"), "-o", out], check=True)
    return out


def test_the_cases_reach_every_kernel(rule):
    lines, want = [], []
    for kernel, counts, h, d in FORWARD:
        P = sum(counts) + LEAD + TAIL
        lines.append(f"0 {P} {len(counts)} {2 * h} {d}")
        want.append(kernel)
    for kernel, counts, h, d in BACKWARD:
        P = sum(counts) + LEAD + TAIL
        lines.append(f"1 {P} {len(counts)} {d} {h}")
        want.append(kernel)
    for kernel, T, h, d in DENSE:
        lines.append(f"0 {T} 1 {2 * h} {d}")
        want.append(kernel)
    got = subprocess.run([rule], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    assert got == want


CHILD = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
L.moe_gated.argtypes = L.moe_gated_dz.argtypes = [P, P, P, P, i32, i64, i64, i64, i64, P, P, P]
L.moe_last_error.restype = ctypes.c_char_p
at = [0x10000000000 + i * (1 << 44) for i in range(5)]  # aligned addresses, far apart, never read
for device in (0, 1, 63, 0):
    stub.stub_set_device(device)
    for line in sys.argv[3:]:
        way, p, e, h, d = line.split(",")
        p, e, h, d = int(p), int(e), int(h), int(d)
        off = at[2] if e > 1 else None
        if way == "fwd":
            st = L.moe_gated(at[0], at[1], None, off, 2, p, e, h, d, at[3], at[4], None)
        else:
            st = L.moe_gated_dz(at[0], at[1], at[3], off, 2, p, e, h, d, at[4], None, None)
        assert st == 0, (line, st, L.moe_last_error())
out = (ctypes.c_int * 3)()
stub.stub_counts(out)
print(*out)
"""


def test_lds_of_every_kernel_on_every_device(L, tmp_path):
    lines = [f"fwd,{sum(c)},{len(c)},{h},{d}" for _, c, h, d in FORWARD]
    lines += [f"dz,{sum(c)},{len(c)},{h},{d}" for _, c, h, d in BACKWARD]
    launches, large, refused = _run(tmp_path, CHILD, *lines)
    assert launches == 4 * len(lines) and large > 0 and refused == 0, (launches, large, refused)

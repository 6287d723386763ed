"""Kernels of more than 64 KB of dynamic LDS on a second device of the same process. The HIP calls are a
stub's (hip_calls_stub.cpp), loaded ahead of the library in a process of its own."""
import os
import subprocess
import sys

import pytest

import moe_ffn_int4_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
L.moe_grouped_matmul.argtypes = L.moe_grouped_matmul_dx.argtypes = [P, P, P, i64, i64, i64, i64, P, i32, P]
L.moe_grouped_matmul_dw.argtypes = [P, P, P, i64, i64, i64, i64, P, i32, i32, P]
L.moe_linear.argtypes = [P, P, P, i32, P, i64, i64, i64, P, i32, P, P]
L.moe_last_error.restype = ctypes.c_char_p
at = [0x10000000000 + i * (1 << 44) for i in range(4)]  # aligned addresses, far apart, never read
for device in (0, 1, 63, 0):
    stub.stub_set_device(device)
    for line in sys.argv[3:]:
        way, p, e, n, k = line.split(",")
        p, e, n, k = int(p), int(e), int(n), int(k)
        if way == "fwd" and e == 1:
            st = L.moe_linear(at[0], at[1], None, 0, None, p, n, k, at[3], 0, None, None)
        elif way == "dw":
            st = L.moe_grouped_matmul_dw(at[0], at[1], at[2], p, e, n, k, at[3], 0, 0, None)
        else:
            fn = L.moe_grouped_matmul if way == "fwd" else L.moe_grouped_matmul_dx
            st = fn(at[0], at[1], at[2], p, e, n, k, at[3], 0, None)
        assert st == 0, (line, st, L.moe_last_error())
out = (ctypes.c_int * 3)()
stub.stub_counts(out)
print(*out)
"""

# each kernel that takes more than 64 KB, each way that it is launched
CASES = ["fwd,1,1,8192,5120", "fwd,4,4,8192,5120",           # streaming, four rows of x
         "fwd,64,16,8192,4096",                              # sixteen
         "fwd,144,1,904,5240", "fwd,144,2,904,5240", "dx,3,1,8704,136", "dw,7195,1,160,80",       # tiles of 32, split
         "fwd,100,1,4096,4096", "fwd,100,2,4096,4096", "dx,17,1,2048,16384", "dw,1600,1,520,520",  # of 64, split
         "fwd,512,1,8192,5120", "fwd,500,2,8192,5120", "dx,512,1,5120,8192", "dw,700,1,1608,1736",  # of 128, four stages
         "fwd,2100,1,2904,2904", "fwd,2100,4,2904,2904", "dx,2100,4,2904,2904", "dw,2100,4,2904,2904"]  # of 256

FORWARD = r"""
import ctypes, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "d", "E", "h")] + [("top_k", i32), ("group_size", i32)]
class Int4(ctypes.Structure):
    _fields_ = [("p", P * 6)]
class Fp8(ctypes.Structure):
    _fields_ = [("p", P * 6), ("act_ub", ctypes.c_float)]
class Shared(ctypes.Structure):
    _fields_ = [("p", P * 3)]
for fn in (L.moe_forward_path, L.moe_forward_fp8):
    fn.argtypes = [P, P, P, P, P, P, P, P, P, i32, P, sz, P]
L.moe_last_error.restype = ctypes.c_char_p
at = [0x10000000000 + i * (1 << 42) for i in range(16)]
dims = Dims(2048, 512, 4, 512, 1, 128)
int4, fp8, shared = Int4((P * 6)(*at[:6])), Fp8((P * 6)(*at[:6]), 0.0), Shared((P * 3)(*at[6:9]))
for device in (0, 1, 63, 0):
    stub.stub_set_device(device)
    for fn, experts in ((L.moe_forward_path, int4), (L.moe_forward_fp8, fp8)):
        st = fn(ctypes.byref(dims), at[9], at[10], None, ctypes.byref(experts), ctypes.byref(shared), at[11], None, None,
                4, at[12], 1 << 40, None)
        assert st == 0, (st, L.moe_last_error())
out = (ctypes.c_int * 3)()
stub.stub_counts(out)
print(*out)
"""


def _run(tmp_path, child, *args):
    """(launches, those of more than 64 KB, those past what their device allows) of `child`."""
    if not os.path.exists(moe.LIB_PATH):
        from moe_ffn_int4_amd import build
        build.build()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("HIP headers not found")
    stub = str(tmp_path / "libstub.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-Wno-attributes", "-o", stub, os.path.join(ROOT, "tests", "hip_calls_stub.cpp")], check=True)
    r = subprocess.run([sys.executable, "-c", child, stub, moe.LIB_PATH, *args], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return map(int, r.stdout.split())


def test_every_device_allows_the_kernels_their_lds(tmp_path):
    launches, large, refused = _run(tmp_path, CHILD, *CASES)
    assert launches == large == 4 * len(CASES), (launches, large)
    assert refused == 0, f"{refused} of {large} launches ask for more LDS than their device allows the kernel"


def test_every_device_allows_the_layer_its_lds(tmp_path):
    """The layer's forward in tiles of 256: int4 and fp8 experts, up and down projections."""
    launches, large, refused = _run(tmp_path, FORWARD)
    assert launches > large >= 4 * 4, (launches, large)
    assert refused == 0, f"{refused} of {large} launches ask for more LDS than their device allows the kernel"

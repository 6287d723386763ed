"""Refusals of the training operators: every bad argument is turned down before any HIP call."""
import pytest
import torch

import moe_ffn_int4_amd as moe

OK, INVALID, WORKSPACE = 0, 1, 4
F = 0x10000000000  # aligned addresses, far apart, never dereferenced


def at(i):
    return F + i * (1 << 44)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from moe_ffn_int4_amd import build
        build.build()
    return moe.lib()


def _said(L):
    return L.moe_last_error().decode()


GROUPED = dict(a=at(0), b=at(1), off=at(2), P=64, E=4, N=128, K=64, out=at(3), fp32=0)


def _grouped(L, which, **kw):
    v = {**GROUPED, **kw}
    args = [v[n] for n in ("a", "b", "off", "P", "E", "N", "K", "out", "fp32")]
    if which == "dw":
        return L.moe_grouped_matmul_dw(*args, 0, None)
    return (L.moe_grouped_matmul if which == "fwd" else L.moe_grouped_matmul_dx)(*args, None)


@pytest.mark.parametrize("which", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("kw,needle", [
    (dict(P=-1), "P = -1"), (dict(P=(1 << 30) + 1), "P ="), (dict(E=0), "E = 0"), (dict(E=257), "E = 257"),
    (dict(N=0), "N = 0"), (dict(N=12), "N = 12"), (dict(K=4), "K = 4"), (dict(K=(1 << 20) + 8), "K ="),
    (dict(E=256, N=1 << 20, K=1 << 20), "1 TiB"), (dict(off=None), "offsets is NULL"), (dict(off=at(2) + 2), "offsets"),
    (dict(a=None), "NULL"), (dict(b=None), "NULL"), (dict(out=None), "NULL"), (dict(a=at(0) + 8), "aligned"),
    (dict(b=at(1) + 2), "aligned"), (dict(out=at(3) + 4), "aligned"), (dict(out=at(0)), "overlaps"),
    (dict(out=at(1) + 16), "overlaps"), (dict(out=at(2)), "overlaps"),
])
def test_grouped_refusals(L, which, kw, needle):
    assert _grouped(L, which, **kw) == INVALID
    assert needle in _said(L), _said(L)


def test_nothing_to_do(L):
    assert _grouped(L, "fwd", P=0) == OK and _grouped(L, "dx", P=0, a=None) == OK
    assert L.moe_linear(None, None, None, 0, None, 0, 64, 64, None, 0, None, None) == OK
    assert L.moe_swiglu(None, 0, 64, None, None) == OK
    assert L.moe_swiglu_backward(None, None, 0, 64, None, None) == OK
    assert L.moe_permute_rows(None, None, 0, 2, 64, None, None) == OK
    assert L.moe_combine(None, 0, None, None, None, 0, 2, 64, None, None) == OK
    assert L.moe_combine_backward(None, None, 0, None, None, 0, 2, 64, None, None, None) == OK


def _linear(L, x=at(0), w=at(1), bias=at(2), act=1, res=at(3), T=64, N=128, K=128, y=at(4), fp32=0, z=at(5)):
    return L.moe_linear(x, w, bias, act, res, T, N, K, y, fp32, z, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(act=5), "act 5"), (dict(act=-1), "act -1"), (dict(T=-1), "P = -1"), (dict(N=20), "N = 20"),
    (dict(x=None), "x is NULL"), (dict(w=None), "w is NULL"), (dict(y=None), "y is NULL"),
    (dict(bias=at(2) + 4), "bias"), (dict(res=at(3) + 2), "residual"), (dict(z=at(5) + 8), "z is not"),
    (dict(y=at(0)), "y overlaps x"), (dict(y=at(3) + 16), "y overlaps residual"), (dict(y=at(2)), "y overlaps bias"),
    (dict(z=at(4)), "overlaps"), (dict(z=at(3)), "z overlaps residual"),
    (dict(y=at(3), fp32=1), "y overlaps residual"),          # in place only where the types agree
    (dict(x=at(3), y=at(3)), "y overlaps x"),                # the residual is x as well
])
def test_linear_refusals(L, kw, needle):
    assert _linear(L, **kw) == INVALID
    assert needle in _said(L), _said(L)


def _dz(L, dy=at(0), z=at(1), act=2, T=64, N=128, dz=at(2), db=at(3), ws=at(4), n=None):
    return L.moe_linear_dz(dy, z, act, T, N, dz, db, ws,
                           L.moe_linear_dz_workspace_bytes(max(T, 0), 128) if n is None else n, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(act=9), INVALID, "act 9"), (dict(N=4), INVALID, "N = 4"), (dict(T=-3), INVALID, "T = -3"),
    (dict(dy=None), INVALID, "dy is NULL"), (dict(z=None), INVALID, "z is NULL"), (dict(dz=None), INVALID, "dz is NULL"),
    (dict(act=0), INVALID, "act none"), (dict(act=0, dz=None, db=None), INVALID, "nothing"),
    (dict(dz=at(0) + 16), INVALID, "dz overlaps dy"), (dict(db=at(0)), INVALID, "db overlaps"),
    (dict(ws=at(2)), INVALID, "workspace overlaps dz"), (dict(ws=at(3)), INVALID, "overlaps"),
    (dict(ws=None), WORKSPACE, "NULL"), (dict(ws=at(4) + 16), WORKSPACE, "256-byte"), (dict(n=16), WORKSPACE, "needs"),
])
def test_linear_dz_refusals(L, kw, code, needle):
    assert _dz(L, **kw) == code
    assert needle in _said(L), _said(L)


def test_linear_dz_workspace(L):
    assert L.moe_linear_dz_workspace_bytes(-1, 64) == 0
    assert L.moe_linear_dz_workspace_bytes(10, 12) == 0
    assert 0 < L.moe_linear_dz_workspace_bytes(0, 8) <= L.moe_linear_dz_workspace_bytes(1 << 30, 8)
    with pytest.raises(ValueError):
        moe.linear_dz_workspace_bytes(4, 7)


@pytest.mark.parametrize("call,needle", [
    (lambda L: L.moe_swiglu(at(0), -1, 64, at(1), None), "rows = -1"),
    (lambda L: L.moe_swiglu(at(0), 4, 60, at(1), None), "h = 60"),
    (lambda L: L.moe_swiglu(None, 4, 64, at(1), None), "z is NULL"),
    (lambda L: L.moe_swiglu(at(0), 4, 64, at(0), None), "y overlaps z"),
    (lambda L: L.moe_swiglu(at(0) + 8, 4, 64, at(1), None), "aligned"),
    (lambda L: L.moe_swiglu_backward(at(0), at(1), 4, 64, at(0), None), "dz overlaps dy"),
    (lambda L: L.moe_swiglu_backward(at(0), at(1), 4, 64, at(1) + 16, None), "dz overlaps z"),
    (lambda L: L.moe_swiglu_backward(at(0), at(1), 4, 64, None, None), "dz is NULL"),
    (lambda L: L.moe_permute_rows(at(0), at(1), 4, 0, 64, at(2), None), "top_k = 0"),
    (lambda L: L.moe_permute_rows(at(0), at(1), 4, 17, 64, at(2), None), "top_k = 17"),
    (lambda L: L.moe_permute_rows(at(0), at(1), 1 << 29, 4, 64, at(2), None), "exceeds 2^30"),
    (lambda L: L.moe_permute_rows(at(0), at(1), 4, 2, 62, at(2), None), "d = 62"),
    (lambda L: L.moe_permute_rows(at(0), at(1), 4, 2, 64, at(0), None), "xp overlaps x"),
    (lambda L: L.moe_permute_rows(at(0), None, 4, 2, 64, at(2), None), "perm is NULL"),
    (lambda L: L.moe_combine(at(0), 0, at(1), at(2), at(3), 4, 2, 64, at(0), None), "y overlaps o"),
    (lambda L: L.moe_combine(at(0), 0, at(1), at(2), at(3), 4, 2, 64, at(3) + 16, None), "y overlaps residual"),
    (lambda L: L.moe_combine(at(0), 0, at(1) + 2, at(2), None, 4, 2, 64, at(4), None), "inv"),
    (lambda L: L.moe_combine(None, 0, at(1), at(2), None, 4, 2, 64, at(4), None), "o is NULL"),
    (lambda L: L.moe_combine_backward(at(0), at(1), 0, at(2), at(3), 4, 2, 64, at(0), at(5), None), "d_o overlaps dy"),
    (lambda L: L.moe_combine_backward(at(0), at(1), 0, at(2), at(3), 4, 2, 64, at(1), at(5), None), "d_o overlaps o"),
    (lambda L: L.moe_combine_backward(at(0), at(1), 0, at(2), at(3), 4, 2, 64, at(4), at(3), None), "d_gates overlaps"),
    (lambda L: L.moe_combine_backward(at(0), None, 0, at(2), at(3), 4, 2, 64, at(4), at(5), None), "o is NULL"),
])
def test_row_refusals(L, call, needle):
    assert call(L) == INVALID
    assert needle in _said(L), _said(L)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: moe.grouped_matmul(x, w, off), lambda: moe.grouped_matmul_dx(x, w, off),
                 lambda: moe.grouped_matmul_dw(x, x, off), lambda: moe.linear(x, w[0]), lambda: moe.linear_dx(x, w[0]),
                 lambda: moe.linear_dw(x, x), lambda: moe.linear_dz(x, x, "silu"), lambda: moe.swiglu(x),
                 lambda: moe.swiglu_backward(x, x), lambda: moe.permute_rows(x, off, 1), lambda: moe.combine(x, off),
                 lambda: moe.combine_backward(x, x, off, off)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.combine(x.half(), off)
    with pytest.raises(ValueError, match="act"):
        moe._act("tanh")


@pytest.mark.parametrize("which", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("kw", [dict(E=256, P=1 << 30, N=8, K=8), dict(E=256, P=1 << 26, N=1 << 20, K=8),
                                dict(E=256, P=1 << 26, N=8, K=1 << 20)])
def test_more_tiles_than_the_kernels_count(L, which, kw):
    """Offsets out of order may make every group all P rows: their tiles have to be countable."""
    spread = {n: F + i * (1 << 52) for i, n in enumerate(("a", "b", "off", "out"))}
    assert _grouped(L, which, **spread, **kw) == INVALID
    assert "too many tiles" in _said(L), _said(L)

"""Gated blocks and their gradient in every kernel against 64 bits.

Bounds. The sums are off by E_s = (R + 1) 2^-23 sum|a b| (train_util). An activation is evaluated to 2^-19 + |e| 2^-21
of its value (the header's; for a slope, of its larger term), e the exponent in it, and its slope is at most 1.13 (1 for none
and relu). So with a = act(g), s = act'(g): y = a u is off by |u| (1.13 E_g + tol |a|) + |a| E_u + their product; dz's
halves dh u s and dh a by |u s| E_dh + |dh u| tol max(1, |s's terms|), |a| E_dh + |dh a| tol. Products of fp32 values add 2^-23 each. One rounding
to bf16 at the end.
"""
import math
import threading

import pytest
import torch

import moe_ffn_int4_amd as moe
from gated_cases import BACKWARD, DENSE, FORWARD, LEAD, TAIL
from train_util import DEV, HALF, U32, offsets_of, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ACTS = list(moe.ACTS)
PAD = 4104  # values around an output: a multiple of 8, of no larger power of two
TINY = 2.0 ** -119  # the header's: smaller magnitudes of an activation may come out as 0


def _inside(shape, fill):
    n = torch.Size(shape).numel()
    buf = torch.full((n + 2 * PAD,), fill, dtype=BF, device=DEV)
    return buf, buf[PAD:PAD + n].view(shape)


def _around(buf, fill):
    return bool((buf[:PAD] == fill).all()) and bool((buf[-PAD:] == fill).all())


def _act(z, act):
    """act(z), act'(z), and by how much of it each may be off, in 64 bits."""
    one, c = torch.ones_like(z), math.sqrt(8 / math.pi)
    if act == "none":
        return z, one, 0.0, 0.0
    if act == "relu":
        return z.clamp(min=0), (z > 0).double(), 0.0, 0.0
    if act == "silu":
        s, e = torch.sigmoid(z), z
        value, terms = z * s, (s, z * s * (1 - s))
    elif act == "gelu":
        s, e = 0.5 * torch.special.erfc(-z / math.sqrt(2)), z * z / 2
        value, terms = z * s, (s, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    else:
        e = c * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(e)
        value, terms = z * s, (s, z * s * (1 - s) * c * (1 + 0.134145 * z * z))
    tol = 2.0 ** -19 + e.abs() * 2.0 ** -21
    return value, terms[0] + terms[1], tol * value.abs() + TINY, tol * torch.maximum(terms[0].abs(), terms[1].abs()) + TINY


def _rounded(ref, err):
    return err + HALF[BF] * (ref.abs() + err)


def _forward_bounds(x, w, bias, act):
    """(y, its bound, z, its bound) of one group."""
    h, R = w.shape[0] // 2, w.shape[1] + 2
    z = x @ w.t()
    size = x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias, size + bias.abs()
    err = (R + 1) * U32 * size
    g, u, eg, eu = z[:, :h], z[:, h:], err[:, :h], err[:, h:]
    a, _, ea, _ = _act(g, act)
    # the activation of the computed g: its slope is at most 1.13, its own error little larger there
    ea = 1.13 * eg + 1.01 * ea
    y = a * u
    ey = u.abs() * ea + a.abs() * eu + ea * eu + U32 * (y.abs() + u.abs() * ea + a.abs() * eu)
    return y, _rounded(y, ey), z, _rounded(z, err)


def _backward_bounds(dy, w2, z, act):
    h = w2.shape[1]
    dh, edh = dy @ w2, (dy.shape[1] + 1) * U32 * (dy.abs() @ w2.abs())
    g, u = z[:, :h], z[:, h:]
    a, s, ea, es = _act(g, act)
    dg, du, y = dh * u * s, dh * a, a * u
    eg = (u * s).abs() * edh + (dh * u).abs() * es + u.abs() * es * edh + 2 * U32 * dg.abs() * 1.01 + 2 * U32 * (dh * u).abs() * es
    eu = a.abs() * edh + dh.abs() * ea + ea * edh + 2 * U32 * du.abs() * 1.01
    ey = u.abs() * ea + U32 * y.abs() * 1.01
    dz = torch.cat([dg, du], 1)
    return dz, _rounded(dz, torch.cat([eg, eu], 1)), y, _rounded(y, ey)


def _rnd(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(BF)


@pytest.mark.parametrize("keep", [True, False], ids=["z", "no-z"])
@pytest.mark.parametrize("i", range(len(FORWARD)), ids=lambda i: "-".join(map(str, FORWARD[i])).replace(" ", ""))
def test_forward(i, keep):
    kernel, counts, h, d = FORWARD[i]
    act = ACTS[i % 5] if keep else ACTS[(i + 2) % 5]
    say(f"gated {kernel} {counts} h={h} d={d} {act} z={keep}")
    g = torch.Generator(device=DEV).manual_seed(i)
    E, P = len(counts), sum(counts) + LEAD + TAIL
    off = offsets_of(counts, LEAD)
    x, w = _rnd(g, P, d), _rnd(g, E, 2 * h, d, scale=1.5 * d ** -0.5)
    ybuf, y = _inside((P, h), 7.0)
    zbuf, z = _inside((P, 2 * h), 5.0) if keep else (None, None)
    got = moe.grouped_gated(x, w, off.to(DEV), act, z=z, out=y)
    assert got is y
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        ref, bound, zref, zbound = _forward_bounds(x[s].double(), w[e].double(), None, act)
        within(y[s], ref, bound, f"y[{e}]")
        if keep:
            within(z[s], zref, zbound, f"z[{e}]")
    # rows of no expert, and what is around
    assert _around(ybuf, 7.0) and bool((y[:LEAD] == 7.0).all()) and bool((y[P - TAIL:] == 7.0).all())
    if keep:
        assert _around(zbuf, 5.0) and bool((z[:LEAD] == 5.0).all()) and bool((z[P - TAIL:] == 5.0).all())
        again = moe.grouped_gated(x, w, off.to(DEV), act)
        assert torch.equal(again[LEAD:P - TAIL], y[LEAD:P - TAIL]), "z changes y"


@pytest.mark.parametrize("kernel,T,h,d,act", [(*c, a) for c in DENSE for a in ACTS if a in ("silu", "gelu") or c[0] in ("stream", "tile64")])
def test_dense_with_bias(kernel, T, h, d, act):
    say(f"gated dense {kernel} {T} {h} {d} {act}")
    g = torch.Generator(device=DEV).manual_seed(T)
    x, w = _rnd(g, T, d), _rnd(g, 2 * h, d, scale=d ** -0.5)
    bias = torch.randn(2 * h, generator=g, device=DEV)
    zbuf, z = _inside((T, 2 * h), 5.0)
    ybuf, y = _inside((T, h), 7.0)
    moe.gated_linear(x, w, bias, act, z=z, out=y)
    ref, bound, zref, zbound = _forward_bounds(x.double(), w.double(), bias.double(), act)
    within(y, ref, bound, "y")
    within(z, zref, zbound, "z")
    assert _around(ybuf, 7.0) and _around(zbuf, 5.0)
    plain = moe.gated_linear(x, w, act=act)
    ref, bound, _, _ = _forward_bounds(x.double(), w.double(), None, act)
    within(plain, ref, bound, "without bias")


@pytest.mark.parametrize("how", ["y", "no-y", "in-place"])
@pytest.mark.parametrize("i", range(len(BACKWARD)), ids=lambda i: "-".join(map(str, BACKWARD[i])).replace(" ", ""))
def test_backward(i, how):
    kernel, counts, h, d = BACKWARD[i]
    act = ACTS[(i + {"y": 0, "no-y": 2, "in-place": 3}[how]) % 5]
    say(f"gated_dz {kernel} {counts} h={h} d={d} {act} {how}")
    g = torch.Generator(device=DEV).manual_seed(i)
    E, P = len(counts), sum(counts) + LEAD + TAIL
    off = offsets_of(counts, LEAD)
    dy, w2, z0 = _rnd(g, P, d), _rnd(g, E, d, h, scale=d ** -0.5), _rnd(g, P, 2 * h, scale=1.5)
    zbuf, z = _inside((P, 2 * h), 5.0)
    z.copy_(z0)
    dbuf, dz = (zbuf, z) if how == "in-place" else _inside((P, 2 * h), 7.0)
    ybuf, y = (None, None) if how == "no-y" else _inside((P, h), 9.0)
    got = moe.grouped_gated_dz(dy, w2, z, off.to(DEV), act, y=y, out=dz)
    assert got is dz
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        ref, bound, yref, ybound = _backward_bounds(dy[s].double(), w2[e].double(), z0[s].double(), act)
        within(dz[s], ref, bound, f"dz[{e}]")
        if y is not None:
            within(y[s], yref, ybound, f"y[{e}]")
    assert _around(dbuf, 5.0 if how == "in-place" else 7.0)
    ends = [slice(0, LEAD), slice(P - TAIL, P)]
    for s in ends:
        assert torch.equal(dz[s], z0[s] if how == "in-place" else torch.full_like(dz[s], 7.0))
        if y is not None:
            assert bool((y[s] == 9.0).all())
    if y is not None:
        assert _around(ybuf, 9.0)
    if how != "in-place":
        assert torch.equal(z, z0) and _around(zbuf, 5.0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,h,d", [(1, 72, 136), (65, 200, 264), (300, 520, 1032)])
def test_dense_backward_against_formula_and_differences(T, h, d, act):
    """The whole way back of a dense gated block with a down-projection: dx, dw, dw2 and bias against autograd in 64 bits,
    and the loss's differences along a direction of each. Values pass at most three roundings to bf16 (z, dz, the gradient; y):
    3 * 2^-8 of the norm, relu's slope changes side where z rounds to another sign."""
    say(f"gated dense backward {T} {h} {d} {act}")
    g = torch.Generator().manual_seed(T + h)
    x, dy = torch.randn(T, d, generator=g).to(BF), torch.randn(T, d, generator=g).to(BF)
    w, w2 = (torch.randn(2 * h, d, generator=g) * d ** -0.5).to(BF), (torch.randn(d, h, generator=g) * h ** -0.5).to(BF)
    b = torch.randn(2 * h, generator=g) * 0.3
    c = [t.to(DEV) for t in (x, w, b, w2, dy)]
    z = torch.empty(T, 2 * h, dtype=BF, device=DEV)
    y = moe.gated_linear(c[0], c[1], c[2], act, z=z)
    again = torch.empty_like(y)
    dz = moe.gated_linear_dz(c[4], c[3], z, act, y=again)
    got = dict(x=moe.linear_dx(dz, c[1]), w=moe.linear_dw(dz, c[0]), b=moe.linear_dz(dz, None)[1], w2=moe.linear_dw(c[4], again))
    q = dict(x=x.double(), w=w.double(), b=b.double(), w2=w2.double())

    def loss(p):
        zz = p["x"] @ p["w"].t() + p["b"]
        zg = zz[:, :h]
        a = {"none": zg, "relu": zg.clamp(min=0), "silu": zg * torch.sigmoid(zg), "gelu": 0.5 * zg * torch.special.erfc(-zg / math.sqrt(2)),
             "gelu_tanh": torch.nn.functional.gelu(zg, approximate="tanh")}[act]
        return (((a * zz[:, h:]) @ p["w2"].t()) * dy.double()).sum()

    leaves = {n: t.clone().requires_grad_(True) for n, t in q.items()}
    grads = dict(zip(q, torch.autograd.grad(loss(leaves), list(leaves.values()))))
    tol = 3 * 2.0 ** -8
    for n, ref in grads.items():
        assert (got[n].double().cpu() - ref).norm() <= tol * ref.norm(), n
        v = torch.randn(ref.shape, generator=g, dtype=torch.float64)
        eps = 1e-6
        want = (loss({**q, n: q[n] + eps * v}) - loss({**q, n: q[n] - eps * v})).item() / (2 * eps)
        along = (got[n].double().cpu() * v).sum().item()
        assert abs(along - want) <= tol * ref.norm().item() * v.norm().item() + 1e-4 * abs(want), n


@pytest.mark.parametrize("act", ACTS)
def test_every_value_of_the_gate(act):
    """A gate at every finite bf16 value (products with the unit matrix are exact), an up factor of 1."""
    v = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(BF)
    v = v[torch.isfinite(v)].to(DEV)
    n = v.numel() // 8 * 8
    z0 = torch.cat([v[:n].reshape(-1, 8), torch.ones(n // 8, 8, dtype=BF, device=DEV)], 1).contiguous()
    ref, slope, ea, es = _act(z0[:, :8].double().clamp(-3e38, 3e38), act)
    eye = torch.eye(16, dtype=BF, device=DEV)
    z = torch.empty_like(z0)
    y = moe.gated_linear(z0, eye, act=act, z=z)
    assert torch.equal(z, z0)
    # past 88 the exponentials are at their limits; the activation is 0 or z there
    near = z0[:, :8].abs() <= 88
    within(torch.where(near, y, 0), torch.where(near, ref, 0.0), torch.where(near, _rounded(ref, ea + U32 * ref.abs()) + 2.0 ** -126, 0.0), "y")
    far = ~near & (z0[:, :8] > 0)
    assert torch.equal(y[far], z0[:, :8][far])
    left = ~near & (z0[:, :8] < 0)
    assert bool(torch.isfinite(y[left]).all()) and (act == "none" or not y[left].any())
    one = torch.ones(n // 8, 8, dtype=BF, device=DEV)
    dz = moe.gated_linear_dz(one, torch.eye(8, dtype=BF, device=DEV), z0, act)
    within(torch.where(near, dz[:, 8:], 0), torch.where(near, ref, 0.0), torch.where(near, _rounded(ref, ea + U32 * ref.abs()) + 2.0 ** -126, 0.0), "dz of u")
    within(torch.where(near, dz[:, :8], 0), torch.where(near, slope, 0.0), torch.where(near, _rounded(slope, es + 4 * U32) + 2.0 ** -126, 0.0), "dz of g")


@pytest.mark.parametrize("P,E", [(5, 2), (40, 1), (700, 3)])
def test_values_that_are_not_finite_stay_in_their_row(P, E):
    g = torch.Generator(device=DEV).manual_seed(P)
    h, d = 264, 520
    off = torch.tensor([0] + [P * (e + 1) // E for e in range(E)], dtype=torch.int32, device=DEV)
    x, w, w2 = _rnd(g, P, d), _rnd(g, E, 2 * h, d, scale=0.05), _rnd(g, E, d, h, scale=0.05)
    clean = moe.grouped_gated(x, w, off)
    x[P // 2, 3] = float("nan")
    y = moe.grouped_gated(x, w, off)
    assert bool(torch.isnan(y[P // 2]).all())
    keep = torch.arange(P, device=DEV) != P // 2
    assert torch.equal(y[keep], clean[keep])
    dy, z = _rnd(g, P, d), _rnd(g, P, 2 * h)
    clean = moe.grouped_gated_dz(dy, w2, z, off)
    dy[P // 2, 5] = float("inf")
    dz = moe.grouped_gated_dz(dy, w2, z, off)
    assert not torch.isfinite(dz[P // 2]).all() and torch.equal(dz[keep], clean[keep])


def test_offsets_that_are_the_callers_mistake():
    """Out of order or out of range: clamped, nothing outside the operands is touched."""
    g = torch.Generator(device=DEV).manual_seed(1)
    P, E, h, d = 300, 4, 136, 264
    x, w, w2, dy, z = _rnd(g, P, d), _rnd(g, E, 2 * h, d), _rnd(g, E, d, h), _rnd(g, P, d), _rnd(g, P, 2 * h)
    for bad in ([0, 200, 100, 250, 300], [-5, 10, 20, 30, 5000], [300, 300, 0, 0, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        ybuf, y = _inside((P, h), 7.0)
        zbuf, zz = _inside((P, 2 * h), 5.0)
        moe.grouped_gated(x, w, off, z=zz, out=y)
        dbuf, dz = _inside((P, 2 * h), 3.0)
        moe.grouped_gated_dz(dy, w2, z, off, out=dz)
        torch.cuda.synchronize()
        assert _around(ybuf, 7.0) and _around(zbuf, 5.0) and _around(dbuf, 3.0)


def test_no_rows():
    w, w2 = torch.ones(2, 32, 16, dtype=BF, device=DEV), torch.ones(2, 16, 16, dtype=BF, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = torch.empty(0, 16, dtype=BF, device=DEV)
    assert moe.grouped_gated(e, w, off).shape == (0, 16)
    assert moe.grouped_gated_dz(e, w2, torch.empty(0, 32, dtype=BF, device=DEV), off).shape == (0, 32)
    # rows, but of no expert
    x = torch.ones(9, 16, dtype=BF, device=DEV)
    y = torch.full((9, 16), 3.0, dtype=BF, device=DEV)
    moe.grouped_gated(x, w, off, out=y)
    assert bool((y == 3.0).all())


def test_streams_threads_and_graphs_give_the_same_bits():
    g = torch.Generator(device=DEV).manual_seed(2)
    cases = []
    for P, E, h, d in ((3, 1, 264, 520), (20, 4, 264, 520), (600, 3, 520, 1032), (2200, 2, 1448, 1032)):
        off = torch.tensor([P * e // E for e in range(E + 1)], dtype=torch.int32, device=DEV)
        cases.append((_rnd(g, P, d), _rnd(g, E, 2 * h, d, scale=0.05), _rnd(g, E, d, h, scale=0.05), _rnd(g, P, d), off))

    def run(c):
        x, w, w2, dy, off = c
        z = torch.empty(x.shape[0], w.shape[1], dtype=BF, device=DEV)
        y = moe.grouped_gated(x, w, off, "gelu", z=z)
        return y, moe.grouped_gated_dz(dy, w2, z, off, "gelu")

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(3):
                for c, ref in zip(cases, want):
                    got = run(c)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, ref)):
                        failed.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for c, ref in zip(cases, want):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = run(c)
        for k in range(3):
            c[0].mul_(-1.0)  # other inputs at each replay
            now = run(c)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, now)), f"replay {k}"


@pytest.mark.parametrize("E,d", [(3, 32768), (1, 65536)])
def test_weights_past_32_bits(E, d):
    """Experts whose weights start past 2^32 bytes, and up rows as far from gate rows as is allowed: 2^32 bytes less 256 rows."""
    h, P = 32768 - 256, 40
    say(f"E={E} h={h} d={d}")
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.empty(E, 2 * h, d, dtype=BF, device=DEV).normal_(0.0, 0.01, generator=g)
    x = _rnd(g, P, d)
    for rows in ((1, 0, 2), (17, 3, 20)) if E == 3 else ((1,), (40,), (300,)):
        if sum(rows) > P:
            x = _rnd(g, sum(rows), d)
        off = offsets_of(rows)
        y = moe.grouped_gated(x, w, off.to(DEV))
        for e in range(E):
            s = slice(int(off[e]), int(off[e + 1]))
            for c in (slice(0, 40), slice(h - 72, h)):
                both = torch.cat([w[e, c], w[e, h + c.start:h + c.stop]])
                ref, bound, _, _ = _forward_bounds(x[s].double(), both.double(), None, "silu")
                within(y[s, c], ref, bound, f"{rows} expert {e} from {c.start}")

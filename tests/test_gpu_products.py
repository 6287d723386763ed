"""grouped_matmul, its gradients and linear against 64-bit products."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, bf16, gen, offsets_of, product_bound, say, split_counts, within

pytestmark = pytest.mark.gpu
OUT = [torch.bfloat16, torch.float32]

# (P, E, N, K, skew, empty groups): one row up to several tiles of every kernel (the
# streaming one, tiles of 64, 128 and 256, blocks that do several tiles, tiles cut in
# two), widths that end inside a tile, a step or a 16-wide sub-tile, groups without rows
SHAPES = [
    (1, 1, 8, 8, 0.0, ()),
    (5, 3, 16, 24, 0.0, (1,)),
    (16, 16, 136, 520, 0.0, ()),
    (64, 4, 512, 256, 0.0, ()),
    (130, 4, 136, 72, 1.0, (0, 3)),
    (257, 12, 264, 200, 1.0, (5,)),
    (300, 256, 64, 64, 0.5, ()),
    (700, 2, 392, 328, 0.0, ()),
    (1500, 5, 776, 1032, 1.0, (2,)),
    (0, 4, 16, 40, 0.0, ()),
    (1500, 2, 1704, 136, 0.0, ()),
    (1500, 2, 136, 1704, 0.0, ()),
    (700, 40, 392, 328, 1.0, (3,)),
    (2100, 3, 2600, 200, 0.5, ()),
    (2100, 3, 200, 2600, 0.5, ()),
    (1300, 3, 1400, 1096, 0.0, ()),
    (9000, 1, 2104, 72, 0.0, ()),
    (9000, 9, 72, 2104, 1.0, (0, 8)),
    (830, 2, 2904, 2904, 0.0, ()),
]
IDS = ["-".join(str(v) for v in s[:4]) for s in SHAPES]


def _case(shape, seed=0):
    P, E, N, K, skew, empty = shape
    g = gen(100 + seed)
    counts = split_counts(P, E, 7 + seed, skew, empty)
    return dict(P=P, E=E, N=N, K=K, counts=counts, off=offsets_of(counts), x=bf16(g, P, K),
                w=bf16(g, E, N, K, scale=0.1), dy=bf16(g, P, N))


def _each(c, fn, shape):
    """fn(rows of each group, e) put together over the groups (rows outside them: 0)."""
    ref = torch.zeros(shape, dtype=torch.float64, device=DEV)
    size = torch.zeros(shape, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        a, b = int(c["off"][e]), int(c["off"][e + 1])
        fn(e, slice(a, b), ref, size)
    return ref.cpu(), size.cpu()


def _wide(t):
    return t.to(DEV).double()


def _fwd(c):
    def one(e, s, ref, size):
        x, w = _wide(c["x"][s]), _wide(c["w"][e]).t()
        ref[s], size[s] = x @ w, x.abs() @ w.abs()
    return _each(c, one, (c["P"], c["N"]))


def _dx(c):
    def one(e, s, ref, size):
        dy, w = _wide(c["dy"][s]), _wide(c["w"][e])
        ref[s], size[s] = dy @ w, dy.abs() @ w.abs()
    return _each(c, one, (c["P"], c["K"]))


def _dw(c):
    def one(e, s, ref, size):
        dy, x = _wide(c["dy"][s]).t(), _wide(c["x"][s])
        ref[e], size[e] = dy @ x, dy.abs() @ x.abs()
    return _each(c, one, (c["E"], c["N"], c["K"]))


def _d(c, *names):
    return [c[n].to(DEV) for n in names]


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, out):
    say(f"grouped_matmul {shape} {out}")
    c = _case(shape)
    y = moe.grouped_matmul(*_d(c, "x", "w", "off"), out_dtype=out)
    assert y.dtype == out
    ref, size = _fwd(c)
    within(y, ref, product_bound(ref, size, c["K"], out), "y")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_dx(shape, out):
    say(f"grouped_matmul_dx {shape} {out}")
    c = _case(shape)
    dx = moe.grouped_matmul_dx(*_d(c, "dy", "w", "off"), out_dtype=out)
    ref, size = _dx(c)
    within(dx, ref, product_bound(ref, size, c["N"], out), "dx")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_dw(shape, out):
    say(f"grouped_matmul_dw {shape} {out}")
    c = _case(shape)
    dw = moe.grouped_matmul_dw(*_d(c, "dy", "x", "off"), out_dtype=out)
    ref, size = _dw(c)
    within(dw, ref, product_bound(ref, size, max(c["counts"] + [0]), out), "dw")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
def test_dw_accumulates(out):
    c = _case(SHAPES[5])
    old = torch.randn(c["E"], c["N"], c["K"], generator=gen(3)).to(out)
    dw = old.to(DEV)
    got = moe.grouped_matmul_dw(*_d(c, "dy", "x", "off"), out=dw, accumulate=True)
    assert got.data_ptr() == dw.data_ptr()
    ref, size = _dw(c)
    within(dw, ref + old.double(),
           product_bound(ref + old.double(), size + old.double().abs(), max(c["counts"]) + 1, out), "dw")
    # a group without rows keeps its values bit for bit
    assert c["counts"][5] == 0 and torch.equal(dw[5].cpu(), old[5])


@pytest.mark.parametrize("rows,N,K", [(40, 264, 136), (300, 264, 136), (1100, 264, 136), (11, 264, 136),
                                      (2000, 2600, 136), (2000, 136, 2600)])
def test_rows_outside_every_group(rows, N, K):
    """Groups that start after row 0 and end before row P: the other rows are neither read
    (NaN there changes nothing) nor written."""
    P, E, lead = rows, 3, 3
    counts = split_counts(P - lead - 5, E, 1)
    off = offsets_of(counts, lead)
    g = gen(4)
    c = dict(P=P, E=E, N=N, K=K, counts=counts, off=off, x=bf16(g, P, K), w=bf16(g, E, N, K), dy=bf16(g, P, N))
    for name in ("x", "dy"):
        c[name][:lead] = float("nan")
        c[name][P - 5:] = float("nan")
    for got, (ref, size), red in [
            (moe.grouped_matmul(*_d(c, "x", "w", "off"), out=torch.full((P, N), 7.0, dtype=torch.bfloat16, device=DEV)),
             _fwd(c), K),
            (moe.grouped_matmul_dx(*_d(c, "dy", "w", "off"), out=torch.full((P, K), 7.0, dtype=torch.bfloat16, device=DEV)),
             _dx(c), N)]:
        ref[:lead], ref[P - 5:] = 7.0, 7.0
        within(got, ref, product_bound(ref, size, red, torch.bfloat16))
        assert bool((got[:lead] == 7).all()) and bool((got[P - 5:] == 7).all())
    ref, size = _dw(c)
    within(moe.grouped_matmul_dw(*_d(c, "dy", "x", "off")), ref, product_bound(ref, size, max(counts), torch.bfloat16))


@pytest.mark.parametrize("P,N,K", [(14, 200, 136), (60, 200, 136), (500, 200, 136), (2500, 2200, 136),
                                   (2500, 136, 2200), (2500, 1104, 1032)])
def test_nan_and_infinity_stay_in_their_rows(P, N, K):
    """A NaN row and an infinite one change only what their formula reads: in y and dx their
    own rows, in dw their own group."""
    c = _case((P, 4, N, K, 0.0, ()))
    bad, inf = int(c["off"][1]), int(c["off"][2])  # first rows of groups 1 and 2
    for name in ("x", "dy"):
        c[name][bad] = float("nan")
        c[name][inf, 3] = float("inf")
    off = c["off"]
    ref, size = _fwd(c)
    within(moe.grouped_matmul(*_d(c, "x", "w", "off")), ref, product_bound(ref, size, c["K"], torch.bfloat16), "y")
    ref, size = _dx(c)
    within(moe.grouped_matmul_dx(*_d(c, "dy", "w", "off")), ref, product_bound(ref, size, c["N"], torch.bfloat16), "dx")
    ref, size = _dw(c)
    dw = moe.grouped_matmul_dw(*_d(c, "dy", "x", "off"))
    within(dw, ref, product_bound(ref, size, max(c["counts"]), torch.bfloat16), "dw")
    assert bool(torch.isfinite(dw[[0, 3]].float()).all()) and int(off[4]) == P


def test_offsets_out_of_range_are_clamped():
    """Bad offsets give wrong or empty groups but no access outside the operands: a range
    past P ends at P, a negative start is 0, a descending pair is empty."""
    P, N, K = 100, 72, 40
    g = gen(9)
    x, w, dy = bf16(g, P, K).to(DEV), bf16(g, 4, N, K).to(DEV), bf16(g, P, N).to(DEV)
    bad = torch.tensor([-5, 20, 10, 90, 1 << 30], dtype=torch.int32, device=DEV)
    y = moe.grouped_matmul(x, w, bad, out=torch.zeros(P, N, dtype=torch.float32, device=DEV))
    dw = moe.grouped_matmul_dw(dy, x, bad)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and bool((dw[1] == 0).all())
    ref = x[90:].double().cpu() @ w[3].double().cpu().t()
    size = x[90:].double().abs().cpu() @ w[3].double().abs().cpu().t()
    within(y[90:], ref, product_bound(ref, size, K, torch.float32))


# ------------------------------------------------------------------- linear

def _act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}[act]()


LINEAR = [(1, 8, 8), (1, 1032, 520), (3, 264, 136), (16, 72, 2056), (17, 72, 2056), (70, 128, 64), (300, 520, 264),
          (1030, 776, 520), (1500, 1704, 136), (3000, 2104, 200)]


@pytest.mark.parametrize("act", list(moe.ACTS))
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(T, N, K, act):
    say(f"linear {T} {N} {K} {act}")
    g = gen(T + N)
    x, w, r = bf16(g, T, K), bf16(g, N, K, scale=K ** -0.5), bf16(g, T, N)
    b = torch.randn(N, generator=g)
    zr = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    for use_bias, use_res, keep_z, out in [(True, True, True, torch.bfloat16), (False, False, False, torch.float32),
                                           (True, False, True, torch.float32), (False, True, False, torch.bfloat16)]:
        pre = zr + b.double() if use_bias else zr
        z = torch.empty(T, N, dtype=torch.bfloat16, device=DEV) if keep_z else None
        y = moe.linear(x.to(DEV), w.to(DEV), b.to(DEV) if use_bias else None, act,
                       r.to(DEV) if use_res else None, z, out_dtype=out)
        ref = _act64(pre, act) + (r.double() if use_res else 0)
        # z's own error, times the slope's largest value (1.13 for gelu), and a few roundings of
        # fp32 in the activation: exp is good to |z| 2^-22
        zerr = (K + 2) * 2.0 ** -23 * (size + b.double().abs())
        aerr = 1.2 * zerr + (pre.abs() + 8) * 2.0 ** -21 * pre.abs() + 2.0 ** -23 * ref.abs()
        within(y, ref, aerr + HALF[out] * (ref.abs() + aerr), f"y {act}")
        if keep_z:
            within(z, pre, zerr + HALF[torch.bfloat16] * (pre.abs() + zerr), "z")


@pytest.mark.parametrize("T", [2, 40, 600])
def test_linear_into_its_residual(T):
    N, K = 264, 136
    g = gen(5)
    x, w, r = bf16(g, T, K).to(DEV), bf16(g, N, K, scale=0.1).to(DEV), bf16(g, T, N).to(DEV)
    apart = moe.linear(x, w, residual=r, act="silu")
    into = moe.linear(x, w, residual=r, act="silu", out=r)
    assert into.data_ptr() == r.data_ptr() and torch.equal(apart, into)


@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear_gradients(T, N, K):
    g = gen(T + K)
    x, w, dz = bf16(g, T, K), bf16(g, N, K, scale=0.1), bf16(g, T, N)
    for out in OUT:
        dx = moe.linear_dx(dz.to(DEV), w.to(DEV), out_dtype=out)
        ref, size = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
        within(dx, ref, product_bound(ref, size, N, out), "dx")
        dw = moe.linear_dw(dz.to(DEV), x.to(DEV), out_dtype=out)
        ref, size = dz.double().t() @ x.double(), dz.double().abs().t() @ x.double().abs()
        within(dw, ref, product_bound(ref, size, T, out), "dw")
        again = dw.clone()
        moe.linear_dw(dz.to(DEV), x.to(DEV), out=again, accumulate=True)
        within(again, dw.double().cpu() + ref, product_bound(2 * ref, 2 * size, T + 1, out) , "dw twice")


# ------------------------------------------------------------ streams, graphs

def _all(c, b, r):
    """Each product once, into tensors of its own."""
    x, w, off, dy = c
    return [moe.grouped_matmul(x, w, off), moe.grouped_matmul_dx(dy, w, off, out_dtype=torch.float32),
            moe.grouped_matmul_dw(dy, x, off), moe.linear(x, w[0], b, "gelu", r),
            moe.linear_dx(dy, w[1]), moe.linear_dw(dy, x, out_dtype=torch.float32)]


@pytest.mark.parametrize("P,N,K", [(12, 264, 136), (600, 264, 136), (2100, 2600, 264)])
def test_two_streams_and_repeats_give_the_same_bits(P, N, K):
    c = _case((P, 4, N, K, 0.5, ()))
    d = _d(c, "x", "w", "off", "dy")
    b, r = torch.randn(N, device=DEV), bf16(gen(1), P, N).to(DEV)
    first = _all(d, b, r)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([_all(d, b, r) for _ in range(3)])
    torch.cuda.synchronize()
    for runs in got:
        for outs in runs:
            for a, e in zip(outs, first):
                assert torch.equal(a, e)


@pytest.mark.parametrize("P,N,K", [(12, 264, 136), (600, 264, 136), (2100, 2600, 264)])
def test_graph_replays_equal_eager(P, N, K):
    cases = [_case((P, 4, N, K, 0.5, ()), seed) for seed in range(3)]
    b, r = torch.randn(N, device=DEV), bf16(gen(1), P, N).to(DEV)
    bufs = _d(cases[0], "x", "w", "off", "dy")
    eager = []
    for c in cases:
        for t, v in zip(bufs, _d(c, "x", "w", "off", "dy")):
            t.copy_(v)
        eager.append([t.clone() for t in _all(bufs, b, r)])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all(bufs, b, r)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = _all(bufs, b, r)
    torch.cuda.synchronize()
    for rep in range(2):
        for c, want in zip(cases, eager):
            for t, v in zip(bufs, _d(c, "x", "w", "off", "dy")):
                t.copy_(v)
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, e in zip(outs, want):
                assert torch.equal(a, e)

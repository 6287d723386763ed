"""SwiGLU, the gradient through an activation, and expert row movement against 64-bit forms."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, U32, bf16, gen, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows and widths around a block's threads, pieces and slices
ROWS = [(1, 8), (3, 64), (5, 72), (33, 520), (130, 2048), (7, 2056), (1, 5000), (300, 16)]


def _sig(z):
    return torch.sigmoid(z)


# exp and the divisions are each good to a few 2^-23, exp to |z| 2^-23 more: 40 covers |z| < 16
# with every product of the formulas
REL = 40 * U32


def _bound(terms, dtype=BF):
    """terms: sum of the absolute values that the formula adds."""
    return REL * terms + HALF[dtype] * (1 + REL) * terms


@pytest.mark.parametrize("rows,h", ROWS)
def test_swiglu(rows, h):
    say(f"swiglu {rows} {h}")
    g = gen(rows + h)
    z, dy = bf16(g, rows, 2 * h, scale=2.0), bf16(g, rows, h)
    a, u, d = z[:, :h].double(), z[:, h:].double(), dy.double()
    y = a * _sig(a) * u
    within(moe.swiglu(z.to(DEV)), y, _bound(y.abs()), "y")
    s = _sig(a)
    dg, du = d * u * (s + a * s * (1 - s)), d * a * s
    size = torch.cat([(d * u).abs() * (s + (a * s * (1 - s)).abs()), du.abs()], 1)
    ref = torch.cat([dg, du], 1)
    within(moe.swiglu_backward(dy.to(DEV), z.to(DEV)), ref, REL * size + HALF[BF] * (ref.abs() + REL * size), "dz")
    zd = z.to(DEV)
    apart = moe.swiglu_backward(dy.to(DEV), zd)
    assert torch.equal(moe.swiglu_backward(dy.to(DEV), zd, out=zd), apart)


def test_swiglu_far_values():
    """Where the sigmoid is 0 or 1 in fp32, and past exp's range."""
    g = torch.tensor([0.0, -0.0, 30.0, -30.0, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38, 1e-30, -1e-30,
                      float("nan"), float("inf"), 5.0, -5.0], dtype=BF)
    u = torch.full_like(g, 2.0)
    z = torch.cat([g, u]).view(1, 32)
    y = moe.swiglu(z.to(DEV)).double().cpu()[0]
    a = g.double()
    ref = a * _sig(a) * 2
    ref[ref.abs() > torch.finfo(BF).max] = float("inf")  # 6e38 rounds to infinity in bf16
    # |exp(-z)| reaches 2^43 at z = -30: exp is off by |z| 2^-23, below -88 the result is under 2^-120
    within(y, ref, (30 + 60) * U32 * ref.abs() + HALF[BF] * ref.abs() + 2.0 ** -110, "y")
    dz = moe.swiglu_backward(torch.ones(1, 16, dtype=BF, device=DEV), z.to(DEV)).double().cpu()[0]
    s = _sig(a)
    slope = torch.where(a.abs() > 90, (a > 0).double(), s + a * s * (1 - s))
    slope[torch.isnan(a)] = float("nan")
    within(dz[:16], 2 * slope, (90 + 90) * U32 * 2 * (s + (a * s * (1 - s)).abs().nan_to_num(0, 0)) + HALF[BF] * 2.2 + 0.0, "dg")
    du = a * _sig(a)
    within(dz[16:], du, 90 * U32 * du.abs() + HALF[BF] * du.abs() + 2.0 ** -110, "du")


def _slope(z, act):
    z = z.clone().requires_grad_(True)
    y = {"relu": lambda: z.clamp(min=0), "silu": lambda: z * _sig(z), "gelu": lambda: z * torch.special.ndtr(z),
         "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}[act]()
    return torch.autograd.grad(y.sum(), z)[0]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,N", [(1, 8), (2, 520), (100, 64), (129, 1032), (1000, 72), (3000, 8), (700, 5120)])
def test_linear_dz(T, N, act):
    say(f"linear_dz {T} {N} {act}")
    g = gen(T + N)
    dy, z = bf16(g, T, N), bf16(g, T, N, scale=2.0)
    slope = _slope(z.double(), act)
    if act == "relu":
        slope = (z.double() > 0).double()
    ref = dy.double() * slope
    err = 40 * U32 * dy.double().abs() * 1.2  # slopes are at most 1.13, their terms below 1.2
    dz, db = moe.linear_dz(dy.to(DEV), z.to(DEV), act)
    within(dz, ref, err + HALF[BF] * (ref.abs() + err), "dz")
    within(db, ref.sum(0), err.sum(0) + (T + 1) * U32 * ref.abs().sum(0), "db")
    for into in ("dy", "z"):
        a, b = dy.to(DEV), z.to(DEV)
        dz2, db2 = moe.linear_dz(a, b, act, out=a if into == "dy" else b)
        assert torch.equal(dz2, dz) and torch.equal(db2, db)


@pytest.mark.parametrize("T,N", [(0, 16), (1, 8), (500, 264)])
def test_linear_dz_without_activation(T, N):
    dy = bf16(gen(2), T, N).to(DEV)
    dz, db = moe.linear_dz(dy, None, "none")
    assert dz is dy
    s = dy.double().cpu()
    within(db, s.sum(0), (T + 1) * U32 * s.abs().sum(0), "db")


def test_linear_dz_far_values():
    z = torch.tensor([[0.0, 1e20, -1e20, 3e38, -3e38, float("inf"), float("-inf"), 100.0]], dtype=BF).to(DEV)
    dy = torch.ones(1, 8, dtype=BF, device=DEV)
    want = {"relu": [0, 1, 0, 1, 0, 1, 0, 1], "silu": [0.5, 1, 0, 1, 0, 1, 0, 1]}
    want["gelu"] = want["gelu_tanh"] = want["silu"]
    for act, w in want.items():
        dz, db = moe.linear_dz(dy, z, act)
        assert dz.float().cpu().tolist() == [[float(v) for v in w]], act
        assert torch.equal(db, dz.float()[0]), act
    nan = torch.full((1, 8), float("nan"), dtype=BF, device=DEV)
    for act in want:
        assert bool(torch.isnan(moe.linear_dz(dy, nan, act)[0]).all()), act


# --------------------------------------------------------- expert row movement

PAIRS = [(1, 1, 8), (4, 3, 72), (33, 8, 520), (257, 2, 2056), (100, 16, 64), (5, 1, 5120)]


def _routing(T, k, seed):
    perm = torch.randperm(T * k, generator=gen(seed)).to(torch.int32)
    inv = torch.empty_like(perm)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32)
    return perm, inv


@pytest.mark.parametrize("T,k,d", PAIRS)
def test_permute_rows(T, k, d):
    perm, _ = _routing(T, k, T)
    x = bf16(gen(1), T, d)
    xp = moe.permute_rows(x.to(DEV), perm.to(DEV), k)
    assert torch.equal(xp.cpu(), x[perm.long() // k])


@pytest.mark.parametrize("o_type", [BF, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,k,d", PAIRS)
def test_combine_and_its_gradient(T, k, d, o_type):
    say(f"combine {T} {k} {d} {o_type}")
    _, inv = _routing(T, k, T)
    g = gen(d)
    o = torch.randn(T * k, d, generator=g).to(o_type)
    gates, r, dy = torch.rand(T, k, generator=g), bf16(g, T, d), bf16(g, T, d)
    rows = o.double()[inv.long()].view(T, k, d)
    for use_g, use_r in [(True, True), (True, False), (False, True), (False, False)]:
        terms = rows * gates.double().unsqueeze(2) if use_g else rows
        ref = terms.sum(1) + (r.double() if use_r else 0)
        err = (k + 1) * U32 * (terms.abs().sum(1) + r.double().abs())
        y = moe.combine(o.to(DEV), inv.view(T, k).to(DEV), gates.to(DEV) if use_g else None,
                        r.to(DEV) if use_r else None)
        within(y, ref, err + HALF[BF] * (ref.abs() + err), "y")
    rd = r.to(DEV)
    flat = moe.combine(o.to(DEV), inv.to(DEV), residual=rd, out=rd, top_k=k)
    assert flat.data_ptr() == rd.data_ptr()
    within(flat, rows.sum(1) + r.double(), (k + 1) * U32 * (rows.abs().sum(1) + r.double().abs()) * 1.01
           + HALF[BF] * (rows.sum(1) + r.double()).abs(), "into residual")
    d_o, dg = moe.combine_backward(dy.to(DEV), o.to(DEV), inv.view(T, k).to(DEV), gates.to(DEV))
    want = torch.empty(T * k, d, dtype=torch.float64)
    want[inv.long()] = (gates.double().unsqueeze(2) * dy.double().unsqueeze(1)).view(T * k, d)
    within(d_o, want, (HALF[BF] + U32) * 1.01 * want.abs(), "d_o")
    prod = dy.double().unsqueeze(1) * rows
    within(dg, prod.sum(2), (d + 1) * U32 * prod.abs().sum(2), "d_gates")


def test_indices_out_of_range_stand_for_zero_rows():
    T, k, d = 6, 2, 72
    x = bf16(gen(1), T, d)
    perm, inv = _routing(T, k, 3)
    perm[4], perm[7] = -1, T * k
    xp = moe.permute_rows(x.to(DEV), perm.to(DEV), k).cpu()
    ok = (perm >= 0) & (perm < T * k)
    assert torch.equal(xp[ok], x[perm[ok].long() // k]) and bool((xp[~ok] == 0).all())
    o = torch.randn(T * k, d, generator=gen(2))
    bad = inv.clone()
    bad[1], bad[10] = -7, 1 << 30
    ok = (bad >= 0) & (bad < T * k)
    terms = torch.where(ok.view(T, k, 1), o.double()[bad.clamp(0, T * k - 1).long()].view(T, k, d), 0.0)
    y = moe.combine(o.to(DEV), bad.view(T, k).to(DEV))
    within(y, terms.sum(1), (k + 1) * U32 * terms.abs().sum(1) + HALF[BF] * terms.sum(1).abs() * 1.01, "y")
    dy = bf16(gen(3), T, d).to(DEV)
    d_o = torch.full((T * k, d), 7.0, dtype=BF, device=DEV)
    _, dg = moe.combine_backward(dy, o.to(DEV), bad.view(T, k).to(DEV), torch.ones(T, k, device=DEV), out=d_o)
    assert dg.view(-1)[1].item() == 0 and dg.view(-1)[10].item() == 0
    for slot in (int(inv[1]), int(inv[10])):  # named by no pair: left as they were
        assert bool((d_o[slot] == 7).all())


def test_no_rows():
    z = torch.empty(0, 32, dtype=BF, device=DEV)
    assert moe.swiglu(z).shape == (0, 16)
    assert moe.swiglu_backward(torch.empty(0, 16, dtype=BF, device=DEV), z).shape == (0, 32)
    i = torch.empty(0, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 16, dtype=BF, device=DEV)
    assert moe.permute_rows(x, i, 2).shape == (0, 16)
    assert moe.combine(x, i.view(0, 2)).shape == (0, 16)
    d_o, dg = moe.combine_backward(x, x, i.view(0, 2), torch.empty(0, 2, device=DEV))
    assert d_o.shape == (0, 16) and dg.shape == (0, 2)


def test_graph_replays_equal_eager():
    T, k, d = 200, 3, 264
    perm, inv = (t.to(DEV) for t in _routing(T, k, 5))
    inv = inv.view(T, k)
    gates = torch.rand(T, k, device=DEV)
    ins = [[bf16(gen(s), T, d), bf16(gen(s + 9), T, 2 * d)] for s in range(2)]
    x, z = (t.to(DEV) for t in ins[0])

    def run():
        xp = moe.permute_rows(x, perm, k)
        y = moe.combine(xp, inv, gates, x)
        return [xp, y, *moe.combine_backward(y, xp, inv, gates), moe.swiglu(z), moe.swiglu_backward(y, z),
                *moe.linear_dz(y, x, "gelu")]

    eager = []
    for a in ins:
        x.copy_(a[0]), z.copy_(a[1])
        eager.append([t.clone() for t in run()])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = run()
    torch.cuda.synchronize()
    for rep in range(2):
        for a, want in zip(ins, eager):
            x.copy_(a[0]), z.copy_(a[1])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for got, e in zip(outs, want):
                assert torch.equal(got, e)

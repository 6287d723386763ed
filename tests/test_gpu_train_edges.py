"""The training operators where calls can go wrong: sums into old values in every kernel, memory
around the outputs, indices named twice, launches of more blocks than a grid row, streams."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, U32, bf16, gen, offsets_of, product_bound, say, split_counts, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
OUT = [torch.bfloat16, torch.float32]

# (P, E, N, K): tiles of 64, of 128 over four stages, of 128 over two, of 256
KERNELS = [(90, 3, 136, 200), (700, 1, 1608, 1736), (700, 40, 392, 328), (2100, 2, 2904, 2904)]


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("P,E,N,K", KERNELS)
def test_dw_accumulates_in_every_kernel(P, E, N, K, out):
    say(f"dw accumulate {P} {E} {N} {K} {out}")
    g = gen(P + N)
    counts = split_counts(P, E, 5)
    off = offsets_of(counts)
    dy, x = bf16(g, P, N).to(DEV), bf16(g, P, K).to(DEV)
    dw = torch.randn(E, N, K, generator=g).to(out).to(DEV)
    old = dw.double()
    moe.grouped_matmul_dw(dy, x, off.to(DEV), out=dw, accumulate=True)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        a, b = dy[s].double().t(), x[s].double()
        ref, size = a @ b + old[e], a.abs() @ b.abs() + old[e].abs()
        within(dw[e], ref, product_bound(ref, size, counts[e] + 1, out), f"dw[{e}]")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("P,E,N,K", [(3, 1, 264, 136), (16, 8, 264, 136), (60, 20, 72, 136)] + KERNELS)
def test_memory_around_the_outputs_is_left(P, E, N, K, out):
    """Outputs that stand inside a larger buffer, 16-byte aligned only: what is around them stays."""
    say(f"around {P} {E} {N} {K} {out}")
    g = gen(P + K)
    off = offsets_of(split_counts(P, E, 6)).to(DEV)
    x, w, dy = bf16(g, P, K).to(DEV), bf16(g, E, N, K, scale=0.1).to(DEV), bf16(g, P, N).to(DEV)
    r, b = bf16(g, P, N).to(DEV), torch.randn(N, generator=g).to(DEV)
    pad = 4104  # values: a multiple of 8, of no larger power of two

    def inside(shape, dtype):
        n = 1
        for v in shape:
            n *= v
        buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[pad:pad + n].view(shape)

    z = inside((P, N), BF)
    for what, shape, call in [
            ("y", (P, N), lambda o: moe.grouped_matmul(x, w, off, out=o)),
            ("dx", (P, K), lambda o: moe.grouped_matmul_dx(dy, w, off, out=o)),
            ("dw", (E, N, K), lambda o: moe.grouped_matmul_dw(dy, x, off, out=o)),
            ("linear", (P, N), lambda o: moe.linear(x, w[0], b, "silu", r, z[1], out=o)),
            ("linear plain", (P, N), lambda o: moe.linear(x, w[0], out=o))]:
        buf, view = inside(shape, out)
        apart = torch.empty(shape, dtype=out, device=DEV)
        call(view)
        assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all()), what
        call(apart)
        assert torch.equal(apart, view), what
    assert bool((z[0][:pad] == 7).all()) and bool((z[0][-pad:] == 7).all())


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("T,N,K", [(500, 1608, 520), (3000, 2104, 200)])
def test_linear_into_its_residual_in_large_tiles(T, N, K, act):
    g = gen(T)
    x, w, r = bf16(g, T, K).to(DEV), bf16(g, N, K, scale=0.1).to(DEV), bf16(g, T, N).to(DEV)
    b = torch.randn(N, generator=g).to(DEV)
    apart = moe.linear(x, w, b, act, r)
    assert torch.equal(moe.linear(x, w, b, act, r, out=r), apart)


@pytest.mark.parametrize("T,k,d", [(9, 5, 72), (40, 7, 264), (130, 6, 1032)])
def test_combine_of_any_number_of_rows(T, k, d):
    g = gen(T)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    o, gates = bf16(g, T * k, d), torch.randn(T, k, generator=g)
    terms = o.double()[inv.long()] * gates.double().unsqueeze(2)
    ref, err = terms.sum(1), (k + 1) * U32 * terms.abs().sum(1)
    within(moe.combine(o.to(DEV), inv.to(DEV), gates.to(DEV)), ref, err + HALF[BF] * (ref.abs() + err), "y")


def test_indices_named_twice():
    """permute_rows and combine read a row as often as it is named; combine_backward writes
    values of one of the pairs that name a row."""
    T, k, d = 50, 4, 136
    g = gen(8)
    x, dy = bf16(g, T, d), bf16(g, T, d)
    perm = torch.randint(0, T * k, (T * k,), generator=g).to(torch.int32)
    assert torch.equal(moe.permute_rows(x.to(DEV), perm.to(DEV), k).cpu(), x[perm.long() // k])
    inv = torch.randint(0, 20, (T, k), generator=g).to(torch.int32)
    o, gates = bf16(g, T * k, d), torch.rand(T, k, generator=g)
    terms = o.double()[inv.long()] * gates.double().unsqueeze(2)
    ref, err = terms.sum(1), (k + 1) * U32 * terms.abs().sum(1)
    within(moe.combine(o.to(DEV), inv.to(DEV), gates.to(DEV)), ref, err + HALF[BF] * (ref.abs() + err), "y")
    d_o = torch.full((T * k, d), 7.0, dtype=BF, device=DEV)
    _, dg = moe.combine_backward(dy.to(DEV), o.to(DEV), inv.to(DEV), gates.to(DEV), out=d_o)
    prod = dy.double().unsqueeze(1) * o.double()[inv.long()]
    within(dg, prod.sum(2), (d + 1) * U32 * prod.abs().sum(2), "d_gates")
    d_o = d_o.cpu()
    each = (gates.unsqueeze(2) * dy.float().unsqueeze(1)).to(BF)
    for slot in range(20):
        named = each[inv == slot]
        assert bool((named == d_o[slot]).any(0).all()), slot
    assert bool((d_o[20:] == 7).all())


def test_more_pairs_than_threads_of_a_grid_row():
    """A wave for each of more than 2^26 pairs."""
    T, k, d = (1 << 22) + 5, 16, 8
    say(f"combine_backward of {T * k} pairs")
    dy = torch.randn(T, d, device=DEV).to(BF)
    gates = torch.rand(T, k, device=DEV)
    inv = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    o = torch.randn(T * k, d, device=DEV, dtype=BF)
    d_o, dg = moe.combine_backward(dy, o, inv, gates)
    # one product in fp32 and one rounding: the same bits
    assert torch.equal(d_o.view(T, k, d), (gates.unsqueeze(2) * dy.float().unsqueeze(1)).to(BF))
    for s in (slice(0, 1000), slice(T - 1000, T)):
        prod = dy[s].double().unsqueeze(1) * o.view(T, k, d)[s].double()
        within(dg[s], prod.sum(2), (d + 1) * U32 * prod.abs().sum(2), "d_gates")


def test_more_blocks_than_a_grid_row():
    # the streaming product: 512 row tiles of 8193 strips
    E, P, N, K = 256, 1024, (1 << 17) + 8, 8
    say(f"grouped_matmul {P} {E} {N} {K}")
    x, w = torch.randn(P, K, device=DEV).to(BF), torch.randn(E, N, K, device=DEV).to(BF)
    off = torch.arange(0, P + 1, 4, dtype=torch.int32, device=DEV)
    y = moe.grouped_matmul(x, w, off)
    for c in (slice(0, 64), slice(N - 200, N)):
        wide = w[:, c].double().transpose(1, 2).contiguous()
        rows = x.double().view(E, 4, K)
        ref, size = torch.bmm(rows, wide).view(P, -1), torch.bmm(rows.abs(), wide.abs()).view(P, -1)
        within(y[:, c], ref, product_bound(ref, size, K, BF), "y")
    del x, w, y
    # rows of five pieces of 256 threads
    rows, h = 1 << 20, 8200
    say(f"swiglu {rows} {h}")
    z = torch.empty(rows, 2 * h, dtype=BF, device=DEV).normal_()
    y = torch.full((rows, h), 7.0, dtype=BF, device=DEV)
    moe.swiglu(z, out=y)
    for s in (slice(0, 300), slice(rows // 2, rows // 2 + 300), slice(rows - 300, rows)):
        assert torch.equal(y[s], moe.swiglu(z[s])), s


def test_row_operators_on_two_streams():
    T, k, d = 300, 4, 520
    g = gen(2)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).to(DEV)
    perm = torch.argsort(inv).to(torch.int32)
    inv = inv.view(T, k)
    x, z, gates = bf16(g, T, d).to(DEV), bf16(g, T, 2 * d).to(DEV), torch.rand(T, k, generator=g).to(DEV)

    def run():
        xp = moe.permute_rows(x, perm, k)
        y = moe.combine(xp, inv, gates, x)
        return [xp, y, *moe.combine_backward(y, xp, inv, gates), moe.swiglu(z), moe.swiglu_backward(y, z),
                *moe.linear_dz(y, x, "silu")]

    first = run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for outs in got:
        for a, e in zip(outs, first):
            assert torch.equal(a, e)


@pytest.mark.parametrize("R", [1024, 1032, 1096, 1160, 2040])
@pytest.mark.parametrize("counts", [(17,), (32,), (33,), (20, 0, 64, 65, 1, 31), (150, 3)])
def test_few_tiles_of_long_reductions(counts, R):
    """The reduction in three parts of a block: steps that divide by three and that do not, row
    tiles of at most 32 rows and of more, a last step that is not whole."""
    P, E, N = sum(counts), len(counts), 136
    g = gen(R + P)
    off = offsets_of(counts)
    x, w = bf16(g, P, R), bf16(g, E, N, R, scale=0.1)
    v = bf16(g, E, R, N, scale=0.1)
    y = moe.grouped_matmul(x.to(DEV), w.to(DEV), off.to(DEV), out_dtype=torch.float32)
    dx = moe.grouped_matmul_dx(x.to(DEV), v.to(DEV), off.to(DEV), out_dtype=torch.float32)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        a = x[s].double()
        for got, b in ((y[s], w[e].double().t()), (dx[s], v[e].double())):
            ref, size = a @ b, a.abs() @ b.abs()
            within(got, ref, product_bound(ref, size, R, torch.float32), f"group {e}")
    if E > 1:
        return
    b, r = torch.randn(N, generator=g), bf16(g, P, N)
    y = moe.linear(x.to(DEV), w[0].to(DEV), b.to(DEV), "relu", r.to(DEV))
    pre = x.double() @ w[0].double().t() + b.double()
    err = (R + 3) * U32 * (x.double().abs() @ w[0].double().abs().t() + b.double().abs() + r.double().abs())
    ref = pre.clamp(min=0) + r.double()
    within(y, ref, err + HALF[BF] * (ref.abs() + err), "linear")


@pytest.mark.parametrize("counts,N,R", [((30,), 6152, 1032), ((300,), 1096, 1000), ((33, 0, 90, 140), 1096, 776),
                                        ((2000,), 264, 8)])
def test_forward_of_long_reductions_and_many_columns(counts, N, R):
    """As above, for outputs too wide for the streaming product; and weight gradients of so many rows."""
    P, E = sum(counts), len(counts)
    g = gen(R + P)
    off = offsets_of(counts)
    x, w, dy = bf16(g, P, R), bf16(g, E, N, R, scale=0.1), bf16(g, P, N)
    y = moe.grouped_matmul(x.to(DEV), w.to(DEV), off.to(DEV))
    dw = moe.grouped_matmul_dw(dy.to(DEV), x.to(DEV), off.to(DEV), out_dtype=torch.float32)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        for got, a, b, red, out in ((y[s], x[s].double(), w[e].double().t(), R, BF),
                                    (dw[e], dy[s].double().t(), x[s].double(), counts[e], torch.float32)):
            ref, size = a @ b, a.abs() @ b.abs()
            within(got, ref, product_bound(ref, size, red, out), f"group {e}")
    if E > 1:
        return
    b, r, z = torch.randn(N, generator=g), bf16(g, P, N), torch.empty(P, N, dtype=BF, device=DEV)
    y = moe.linear(x.to(DEV), w[0].to(DEV), b.to(DEV), "relu", r.to(DEV), z, out_dtype=torch.float32)
    pre = x.double() @ w[0].double().t() + b.double()
    err = (R + 3) * U32 * (x.double().abs() @ w[0].double().abs().t() + b.double().abs() + r.double().abs())
    ref = pre.clamp(min=0) + r.double()
    within(y, ref, err + HALF[torch.float32] * (ref.abs() + err), "linear")
    within(z, pre, err + HALF[BF] * (pre.abs() + err), "z")


@pytest.mark.parametrize("counts,N,K", [((1,), 65568, 2056), ((3, 0, 1, 9, 4, 0, 2, 5), 9000, 2320),
                                        ((16,), 66000, 2568), ((2, 0, 7), 32776, 3080)])
def test_streaming_blocks_of_several_strips(counts, N, K):
    """More strips of weight rows than blocks: a wave's ring goes on from strip to strip and from
    group to group; waves of unequal numbers of chunks, a last chunk and strip that are not whole."""
    P, E = sum(counts), len(counts)
    say(f"streaming {counts} {N} {K}")
    off = offsets_of(counts)
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(P, K, generator=g, device=DEV).to(BF)
    w = torch.randn(E, N, K, generator=g, device=DEV).mul_(0.1).to(BF)
    y = moe.grouped_matmul(x, w, off.to(DEV))
    b, r = torch.randn(N, generator=g, device=DEV), torch.randn(P, N, generator=g, device=DEV).to(BF)
    lin = moe.linear(x, w[0], b, "relu", r) if E == 1 else None
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if counts[e] == 0:
            continue
        a, c = x[s].double(), w[e].double().t()
        ref, size = a @ c, a.abs() @ c.abs()
        within(y[s], ref, product_bound(ref, size, K, BF), f"group {e}")
        if lin is not None:
            err = (K + 3) * U32 * (size + b.double().abs() + r.double().abs())
            ref = (ref + b.double()).clamp(min=0) + r.double()
            within(lin, ref, err + HALF[BF] * (ref.abs() + err), "linear")


@pytest.mark.parametrize("P,E,N,K", [(3, 4, 264, 136), (14, 4, 8200, 2056)] + [(P, 4, N, K) for P, _, N, K in KERNELS]
                         + [(2100, 4, 2600, 200)])
def test_offsets_out_of_order_stay_inside(P, E, N, K):
    """Nothing outside the operands is written, and what is written comes from the operands."""
    say(f"offsets out of order {P} {E} {N} {K}")
    g = gen(P)
    off = torch.tensor([0, P, P // 2, 3 * P, -7], dtype=torch.int32, device=DEV)
    x, w, dy = bf16(g, P, K).to(DEV), bf16(g, E, N, K, scale=0.1).to(DEV), bf16(g, P, N).to(DEV)
    pad = 4096
    for what, n, call in [("y", P * N, lambda o: moe.grouped_matmul(x, w, off, out=o.view(P, N))),
                          ("dx", P * K, lambda o: moe.grouped_matmul_dx(dy, w, off, out=o.view(P, K))),
                          ("dw", E * N * K, lambda o: moe.grouped_matmul_dw(dy, x, off, out=o.view(E, N, K)))]:
        buf = torch.full((n + 2 * pad,), 7.0, device=DEV)
        call(buf[pad:pad + n])
        assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all()), what
        assert bool(torch.isfinite(buf).all()), what


@pytest.mark.parametrize("counts,N,R", [((30,), 9000, 1032), ((1000,), 552, 1000), ((900, 800), 1000, 776)])
def test_many_columns_of_long_reductions(counts, N, R):
    """Outputs of more tiles than one kernel's split takes and fewer than the next needs, each direction."""
    P, E = sum(counts), len(counts)
    g = gen(R + N)
    off = offsets_of(counts)
    x, w, v, dy = bf16(g, P, R), bf16(g, E, N, R, scale=0.1), bf16(g, E, R, N, scale=0.1), bf16(g, P, N)
    y = moe.grouped_matmul(x.to(DEV), w.to(DEV), off.to(DEV), out_dtype=torch.float32)
    dx = moe.grouped_matmul_dx(x.to(DEV), v.to(DEV), off.to(DEV))
    dw = moe.grouped_matmul_dw(dy.to(DEV), x.to(DEV), off.to(DEV))
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        for got, a, b, red, out in ((y[s], x[s].double(), w[e].double().t(), R, torch.float32),
                                    (dx[s], x[s].double(), v[e].double(), R, BF),
                                    (dw[e], dy[s].double().t(), x[s].double(), counts[e], BF)):
            ref, size = a @ b, a.abs() @ b.abs()
            within(got, ref, product_bound(ref, size, red, out), f"group {e}")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("P,E,N,K", [(600, 1, 72, 88), (1300, 2, 136, 40), (5000, 1, 8, 8)])
def test_dw_accumulates_over_long_reductions(P, E, N, K, out):
    g = gen(P + N)
    counts = split_counts(P, E, 5)
    off = offsets_of(counts)
    dy, x = bf16(g, P, N).to(DEV), bf16(g, P, K).to(DEV)
    dw = torch.randn(E, N, K, generator=g).to(out).to(DEV)
    old = dw.double()
    moe.grouped_matmul_dw(dy, x, off.to(DEV), out=dw, accumulate=True)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        a, b = dy[s].double().t(), x[s].double()
        ref, size = a @ b + old[e], a.abs() @ b.abs() + old[e].abs()
        within(dw[e], ref, product_bound(ref, size, counts[e] + 1, out), f"dw[{e}]")


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("T,N", [(511, 72), (512, 8), (513, 72), (512, 1000), (65, 136), (129, 8192), (600, 64)])
def test_linear_dz_around_its_kernels(T, N, act):
    """Rows around one launch's; a buffer around dz and db that stays; in place; without db (through C)."""
    g = gen(T + N)
    dy, z = bf16(g, T, N), bf16(g, T, N, scale=2.0)
    zz = z.double()
    s = torch.sigmoid(zz)
    slope = s + zz * s * (1 - s) if act == "silu" else torch.ones_like(zz)
    ref = dy.double() * slope
    err = 40 * U32 * dy.double().abs() * 1.2
    pad = 128
    dbuf = torch.full((N + 2 * pad,), 7.0, device=DEV)
    zbuf = torch.full((T * N + 2 * pad,), 7.0, dtype=BF, device=DEV)
    out = zbuf[pad:-pad].view(T, N) if act != "none" else None
    dz, db = moe.linear_dz(dy.to(DEV), z.to(DEV) if act != "none" else None, act, out=out, db=dbuf[pad:-pad])
    within(db, ref.sum(0), err.sum(0) + (T + 1) * U32 * ref.abs().sum(0), "db")
    assert bool((dbuf[:pad] == 7).all()) and bool((dbuf[-pad:] == 7).all())
    if act == "none":
        return
    within(dz, ref, err + HALF[BF] * (ref.abs() + err), "dz")
    assert bool((zbuf[:pad] == 7).all()) and bool((zbuf[-pad:] == 7).all())
    a = dy.to(DEV)
    d2, db2 = moe.linear_dz(a, z.to(DEV), act, out=a)
    assert torch.equal(d2, dz) and torch.equal(db2, db)
    a, b, c = dy.to(DEV), z.to(DEV), torch.empty(T, N, dtype=BF, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert moe.lib().moe_linear_dz(a.data_ptr(), b.data_ptr(), moe.ACTS[act], T, N, c.data_ptr(), None, None, 0, stream) == 0
    assert torch.equal(c, dz)


def test_calls_from_several_threads():
    """Four threads, each with a stream of its own, call every operator at once; one of
    them also makes calls that are refused, whose text the others do not see."""
    import threading
    T, k, d, h, E = 96, 2, 264, 136, 4
    g = gen(12)
    perm = torch.randperm(T * k, generator=g).to(torch.int32)
    inv = torch.empty_like(perm)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32)
    off = offsets_of(split_counts(T * k, E, 3)).to(DEV)
    perm, inv = perm.to(DEV), inv.view(T, k).to(DEV)
    x, gates = bf16(g, T, d).to(DEV), torch.rand(T, k, generator=g).to(DEV)
    w13, w2 = bf16(g, E, 2 * h, d, scale=0.1).to(DEV), bf16(g, E, d, h, scale=0.1).to(DEV)
    s1, b1 = bf16(g, h, d, scale=0.1).to(DEV), torch.randn(h, generator=g).to(DEV)

    def run():
        xp = moe.permute_rows(x, perm, k)
        z = moe.grouped_matmul(xp, w13, off)
        hid = moe.swiglu(z)
        o = moe.grouped_matmul(hid, w2, off)
        y = moe.combine(o, inv, gates, residual=x)
        d_o, dg = moe.combine_backward(y, o, inv, gates)
        dz = moe.swiglu_backward(moe.grouped_matmul_dx(d_o, w2, off), z)
        pre = torch.empty(T, h, dtype=BF, device=DEV)
        a = moe.linear(x, s1, b1, "gelu", z=pre)
        da, db = moe.linear_dz(a, pre, "gelu")
        return [xp, z, hid, o, y, d_o, dg, dz, a, da, db, moe.grouped_matmul_dw(d_o, hid, off),
                moe.grouped_matmul_dw(dz, xp, off, out_dtype=torch.float32), moe.linear_dx(da, s1), moe.linear_dw(da, x)]

    want = run()
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for rep in range(5):
                    got[i, rep] = run()
                    if i == 0:
                        with pytest.raises(moe.MoEError, match="overlaps"):
                            moe.swiglu(want[1], out=want[1].view(-1)[:T * k * h].view(T * k, h))
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: B036 -- shown by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    assert len(got) == 20
    for outs in got.values():
        for a, b in zip(outs, want):
            assert torch.equal(a, b)

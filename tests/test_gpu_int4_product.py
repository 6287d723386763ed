"""Products with 4-bit weights against 64 bits.

Bound. A group's sum is formed of x (code + 24), at most 31 |x|, and of 24 |x|: 55 sum|x| at most, over 130 additions off by
2^-23 each; times the scale. The groups' sums are added in fp32, one rounding for each group, part and epilogue step, of
sum |x code scale|, bias and residual. Activations: the header's 2^-19 + |e| 2^-21 of the value, slope at most 1.13.
"""
import math
import threading

import pytest
import torch

import moe_ffn_int4_amd as moe
from int4_cases import DENSE, GROUPED, LEAD, TAIL
from test_gpu_gated import _act
from train_util import DEV, HALF, U32, offsets_of, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
OUT = [torch.bfloat16, torch.float32]
PAD = 4112  # values around an output


def _inside(shape, dtype, fill):
    n = torch.Size(shape).numel()
    buf = torch.full((n + 2 * PAD,), fill, dtype=dtype, device=DEV)
    return buf, buf[PAD:PAD + n].view(shape)


def _around(buf, fill):
    return bool((buf[:PAD] == fill).all()) and bool((buf[-PAD:] == fill).all())


def _weights(g, E, N, K, group):
    """Tiled codes and scales [E, ...], and codes [E, N, K] and scales [E, N, K / group] as numbers."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randn(E, N, K // group, generator=g, device=DEV) * 0.01  # of either sign
    s[:, ::7, 0] = 0.0
    tiled = [moe.tile_int4(q[e], s[e], group) for e in range(E)]
    return torch.stack([t[0] for t in tiled]), torch.stack([t[1] for t in tiled]), moe.unpack_int4(q).double(), s.double()


def _product(x, codes, scales, group):
    """x w^T and its bound before the epilogue, and sum |x w|."""
    wide = scales.repeat_interleave(group, dim=1)
    ref = x @ (codes * wide).t()
    size = x.abs() @ (codes * wide).abs().t()
    err = U32 * (131 * 55 * (x.abs() @ wide.abs().t()) + (scales.shape[1] + 8) * size)
    return ref, err


def _x(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("i", range(len(GROUPED)), ids=lambda i: "-".join(map(str, GROUPED[i])).replace(" ", ""))
def test_grouped(i, group):
    shape, counts, N, K = GROUPED[i]
    say(f"int4 {shape} {counts} {N} {K} group {group}")
    g = torch.Generator(device=DEV).manual_seed(i)
    E, P = len(counts), sum(counts) + LEAD + TAIL
    off = offsets_of(counts, LEAD)
    q, s, codes, scales = _weights(g, E, N, K, group)
    x = _x(g, P, K)
    for out in OUT:
        buf, y = _inside((P, N), out, 7.0)
        assert moe.grouped_matmul_int4(x, q, s, off.to(DEV), out=y) is y
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            ref, err = _product(x[r].double(), codes[e], scales[e], group)
            within(y[r], ref, err + HALF[out] * (ref.abs() + err), f"{out} y[{e}]")
        assert _around(buf, 7.0) and bool((y[:LEAD] == 7.0).all()) and bool((y[P - TAIL:] == 7.0).all())


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("i", range(len(DENSE)), ids=lambda i: "-".join(map(str, DENSE[i])))
def test_dense(i, group):
    shape, T, N, K = DENSE[i]
    say(f"int4 dense {shape} {T} {N} {K} group {group}")
    g = torch.Generator(device=DEV).manual_seed(T + N)
    q, s, codes, scales = _weights(g, 1, N, K, group)
    x, bias, res = _x(g, T, K), torch.randn(N, generator=g, device=DEV), _x(g, T, N)
    ref, err = _product(x.double(), codes[0], scales[0], group)
    for k, act in enumerate(moe.ACTS):
        out = OUT[(i + k) % 2]
        b, r = (bias if k % 2 else None), (res if k in (0, 3, 4) else None)
        z = ref + b.double() if b is not None else ref
        ez = err + U32 * z.abs()
        v, _, ea, _ = _act(z, act)
        e = 1.13 * ez + 1.01 * ea
        if r is not None:
            v = v + r.double()
            e = e + U32 * v.abs()
        buf, y = _inside((T, N), out, 7.0)
        moe.linear_int4(x, q[0], s[0], b, act, r, out=y)
        within(y, v, e + HALF[out] * (v.abs() + e), f"{act} {out}")
        assert _around(buf, 7.0)
        if r is not None and out == BF:
            same = r.clone()
            assert torch.equal(moe.linear_int4(x, q[0], s[0], b, act, same, out=same), y), "into the residual"


def test_weights_that_the_quantizer_wrote():
    """quantize_int4 to linear_int4: a step of the code at most from the product of the fp32 weights."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for group in moe.GROUPS:
        w = torch.randn(272, 1152, generator=g, device=DEV) * 0.05
        q, s = moe.quantize_int4(w, tiled=True, group=group)
        rq, rs = moe.quantize_int4(w, group=group)
        codes = moe.unpack_int4(rq).double()
        assert torch.equal(moe.unpack_int4(moe.untile_int4(q, 272, 1152)).double(), codes)
        for T in (1, 9, 70):
            x = _x(g, T, 1152)
            ref, err = _product(x.double(), codes, rs.double(), group)
            within(moe.linear_int4(x, q, s, out_dtype=torch.float32), ref, err + HALF[torch.float32] * ref.abs(), f"{group} {T}")
            # the quantizer's own error: half a step, a whole one at +8, where the code ends at 7
            off = x.double().abs() @ rs.double().repeat_interleave(group, 1).t()
            assert bool(((x.double() @ w.double().t() - ref).abs() <= off * 1.01).all())


def test_extreme_codes():
    """All codes -8, all 7, and x of one sign: the sums that cancel are largest."""
    K, N = 4096, 64
    for byte, code in ((0x88, -8), (0x77, 7), (0x00, 0), (0xFF, -1)):
        q = torch.full((N, K // 2), byte, dtype=torch.uint8, device=DEV)
        s = torch.full((N, K // 128), 0.01, device=DEV)
        codes = torch.full((N, K), float(code), dtype=torch.float64, device=DEV)
        for T in (1, 20, 600):
            x = (torch.rand(T, K, generator=torch.Generator(device=DEV).manual_seed(T), device=DEV) + 0.5).to(BF)
            ref, err = _product(x.double(), codes, s.double(), 128)
            within(moe.linear_int4(x, q, s, out_dtype=torch.float32), ref, err + HALF[torch.float32] * ref.abs(), f"{code} {T}")


@pytest.mark.parametrize("T", [3, 15, 31, 60, 300, 700])
def test_values_that_are_not_finite_stay_in_their_row(T):
    g = torch.Generator(device=DEV).manual_seed(T)
    q, s, _, _ = _weights(g, 1, 144, 512, 64)
    x = _x(g, T, 512)
    clean = moe.linear_int4(x, q[0], s[0])
    for bad in (float("nan"), float("inf")):
        x[T // 2, 77] = bad
        y = moe.linear_int4(x, q[0], s[0])
        keep = torch.arange(T, device=DEV) != T // 2
        assert torch.equal(y[keep], clean[keep])
        assert bool(torch.isnan(y[T // 2]).all())


def test_large_and_tiny_rows():
    """|x| up to the header's 2^110, and rows of subnormal products."""
    g = torch.Generator(device=DEV).manual_seed(5)
    q, s, codes, scales = _weights(g, 1, 64, 256, 128)
    for p in (109, -60, -100):
        x = (torch.randn(7, 256, generator=g, device=DEV).clamp(-1.9, 1.9) * 2.0 ** p).to(BF)
        ref, err = _product(x.double(), codes[0], scales[0], 128)
        within(moe.linear_int4(x, q[0], s[0], out_dtype=torch.float32), ref, err + HALF[torch.float32] * ref.abs() + 2.0 ** -126, f"2^{p}")


def test_offsets_that_are_the_callers_mistake():
    g = torch.Generator(device=DEV).manual_seed(1)
    q, s, _, _ = _weights(g, 4, 144, 256, 128)
    for P in (9, 300):
        x = _x(g, P, 256)
        for bad in ([0, P, P // 2, P, P], [-5, 1, 2, 3, 5000], [P, P, 0, 0, 0]):
            buf, y = _inside((P, 144), BF, 7.0)
            moe.grouped_matmul_int4(x, q, s, torch.tensor(bad, dtype=torch.int32, device=DEV), out=y)
            torch.cuda.synchronize()
            assert _around(buf, 7.0)


def test_no_rows():
    q, s = torch.zeros(2, 32, 64, dtype=torch.uint8, device=DEV), torch.ones(2, 32, 1, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe.grouped_matmul_int4(torch.empty(0, 128, dtype=BF, device=DEV), q, s, off).shape == (0, 32)
    assert moe.linear_int4(torch.empty(0, 128, dtype=BF, device=DEV), q[0], s[0]).shape == (0, 32)
    y = torch.full((9, 32), 3.0, dtype=BF, device=DEV)
    moe.grouped_matmul_int4(torch.ones(9, 128, dtype=BF, device=DEV), q, s, off, out=y)
    assert bool((y == 3.0).all())


def test_streams_threads_and_graphs_give_the_same_bits():
    g = torch.Generator(device=DEV).manual_seed(2)
    cases = []
    for P, E, N, K, group in ((1, 1, 272, 640, 128), (9, 4, 144, 1152, 32), (40, 2, 144, 1152, 64), (300, 2, 272, 640, 128), (1500, 2, 272, 640, 128)):
        q, s, _, _ = _weights(g, E, N, K, group)
        cases.append((_x(g, P, K), q, s, torch.tensor([P * e // E for e in range(E + 1)], dtype=torch.int32, device=DEV)))

    def run(c):
        return moe.grouped_matmul_int4(*c), moe.linear_int4(c[0], c[1][0], c[2][0], act="gelu")

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
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
    for c in cases:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = run(c)
        for k in range(3):
            c[0].mul_(-0.5)
            now = run(c)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, now)), f"replay {k}"


def test_weights_past_32_bits():
    """An expert whose codes start past 2^32 bytes, for each kind of tile."""
    E, N, K, group = 3, 65536, 65536, 128
    say(f"E={E} N={N} K={K}")
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(E, N, K // group, generator=g, device=DEV)
    for rows in ((1, 0, 2), (7, 3, 20), (70, 0, 80)):
        off = offsets_of(rows)
        x = _x(g, sum(rows), K)
        y = moe.grouped_matmul_int4(x, q, s, off.to(DEV), out_dtype=torch.float32)
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            for c in (slice(0, 32), slice(N - 48, N)):
                n = c.stop - c.start
                codes = moe.unpack_int4(moe.untile_int4(q[e, c], n, K)).double()
                scales = moe.untile_scales(s[e, c], n, K, group).double()
                ref, err = _product(x[r].double(), codes, scales, group)
                within(y[r, c], ref, err + HALF[torch.float32] * ref.abs(), f"{rows} expert {e} from {c.start}")


def test_binding_refusals():
    q, s, x = torch.zeros(32, 64, dtype=torch.uint8, device=DEV), torch.ones(32, 1, device=DEV), torch.ones(2, 128, dtype=BF, device=DEV)
    off = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    for bad in (lambda: moe.linear_int4(x[:, :64].contiguous(), q, s), lambda: moe.linear_int4(x, q, s[:16]), lambda: moe.linear_int4(x, q, s.expand(32, 3).contiguous()),
                lambda: moe.linear_int4(x, q.cpu(), s), lambda: moe.grouped_matmul_int4(x, q, s, off), lambda: moe.linear_int4(x, q[None], s[None]),
                lambda: moe.linear_int4(x, q, s, act="tanh"), lambda: moe.grouped_matmul_int4(x, q[None], s[None], off[:1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        moe.linear_int4(x, q.to(torch.int8), s)
    assert math.isfinite(moe.linear_int4(x, q, s).float().sum().item())

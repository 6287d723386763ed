"""The product kernels at sizes that the rule sends to each of them, against 64-bit products."""
import threading

import pytest
import torch

import moe_ffn_int4_amd as moe
from matmul_cases import GROUPED, LEAD, LINEAR, TAIL
from train_util import DEV, HALF, offsets_of, product_bound, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
OUT = [torch.bfloat16, torch.float32]
CASES = [(kernel, *case) for kernel, cases in GROUPED.items() for case in cases]
IDS = ["-".join([k, way, *map(str, counts), str(N), str(K)]) for k, way, counts, N, K in CASES]
PAD = 4104  # values around an output: a multiple of 8, of no larger power of two


def _inside(shape, dtype, fill):
    """A buffer of `fill` and, in its middle, a tensor of `shape`, 16-byte aligned only."""
    n = torch.Size(shape).numel()
    buf = torch.full((n + 2 * PAD,), fill, dtype=dtype, device=DEV)
    return buf, buf[PAD:PAD + n].view(shape)


def _around(buf, fill):
    return bool((buf[:PAD] == fill).all()) and bool((buf[-PAD:] == fill).all())


def _operands(way, counts, N, K):
    """The call's operands and, for each group, its slice of the output and its two 64-bit factors."""
    g = torch.Generator(device=DEV).manual_seed(sum(counts) + N)
    E, P = len(counts), sum(counts) + LEAD + TAIL
    off = offsets_of(counts, LEAD)

    def rnd(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(BF)

    a = rnd(P, K if way == "fwd" else N)
    b = rnd(P, K) if way == "dw" else rnd(E, N, K, scale=0.1)
    rows = [slice(int(off[e]), int(off[e + 1])) for e in range(E)]
    return a, b, off.to(DEV), rows


def _call(way, a, b, off, out, **kw):
    return {"fwd": moe.grouped_matmul, "dx": moe.grouped_matmul_dx, "dw": moe.grouped_matmul_dw}[way](a, b, off, out=out, **kw)


def _factors(way, a, b, s, e):
    if way == "dw":
        return a[s].double().t(), b[s].double()
    return a[s].double(), b[e].double().t() if way == "fwd" else b[e].double()


def _check(way, a, b, rows, got, out, N, K, old=None):
    for e, s in enumerate(rows):
        at = e if way == "dw" else s
        x, y = _factors(way, a, b, s, e)
        red = s.stop - s.start if way == "dw" else K if way == "fwd" else N
        if x.numel() == 0 and way != "dw":
            continue
        ref, size = x @ y, x.abs() @ y.abs()
        if old is not None:
            ref, size, red = ref + old[e], size + old[e].abs(), red + 1
        within(got[at], ref, product_bound(ref, size, red, out), f"group {e}")


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("kernel,way,counts,N,K", CASES, ids=IDS)
def test_products(kernel, way, counts, N, K, out):
    """Every value; rows outside the groups hold NaN, which changes nothing, and their rows of the
    output and the memory around it stay. (An empty group's weight gradient is zeros.)"""
    say(f"{kernel} {way} {counts} {N} {K} {out}")
    a, b, off, rows = _operands(way, counts, N, K)
    for t in (a, b) if way == "dw" else (a,):
        t[:LEAD] = float("nan")
        t[-TAIL:] = float("nan")
    shape = (len(counts), N, K) if way == "dw" else (a.shape[0], N if way == "fwd" else K)
    buf, view = _inside(shape, out, 7.0)
    _call(way, a, b, off, view)
    _check(way, a, b, rows, view, out, N, K)
    assert _around(buf, 7.0)
    if way != "dw":
        assert bool((view[:LEAD] == 7).all()) and bool((view[-TAIL:] == 7).all())


@pytest.mark.parametrize("kernel,way,counts,N,K", CASES, ids=IDS)
def test_nan_and_infinity(kernel, way, counts, N, K):
    """A NaN row of one group and an infinite value in another's change only what reads them."""
    say(f"{kernel} {way} {counts} {N} {K}: NaN, infinity")
    a, b, off, rows = _operands(way, counts, N, K)
    filled = [s for s in rows if s.stop > s.start]
    a[filled[0].stop - 1] = float("nan")
    a[filled[-1].start, 3] = float("inf")
    shape = (len(counts), N, K) if way == "dw" else (a.shape[0], N if way == "fwd" else K)
    got = _call(way, a, b, off, torch.full(shape, 7.0, device=DEV))
    _check(way, a, b, rows, got, torch.float32, N, K)


DW = [c for c in CASES if c[1] == "dw"]


@pytest.mark.parametrize("out", OUT, ids=["bf16", "fp32"])
@pytest.mark.parametrize("kernel,way,counts,N,K", DW, ids=[i for i, c in zip(IDS, CASES) if c[1] == "dw"])
def test_weight_gradients_are_added(kernel, way, counts, N, K, out):
    say(f"{kernel} dw {counts} {N} {K} {out}: accumulate")
    a, b, off, rows = _operands(way, counts, N, K)
    buf, view = _inside((len(counts), N, K), out, 7.0)
    view.copy_(torch.randn(view.shape, device=DEV))
    first = view.clone()
    _call(way, a, b, off, view, accumulate=True)
    _check(way, a, b, rows, view, out, N, K, old=first.double())
    for e, n in enumerate(counts):
        assert n > 0 or torch.equal(view[e], first[e])  # bit for bit
    assert _around(buf, 7.0)


LINEARS = [(kernel, *case) for kernel, cases in LINEAR.items() for case in cases]


def _act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}[act]()


@pytest.mark.parametrize("act", list(moe.ACTS))
@pytest.mark.parametrize("kernel,T,N,K", LINEARS)
def test_linear(kernel, T, N, K, act):
    """Bias, activation, residual (also in place) and z, alone and together."""
    say(f"{kernel} linear {T} {N} {K} {act}")
    g = torch.Generator(device=DEV).manual_seed(T + N)
    x, w = torch.randn(T, K, generator=g, device=DEV).to(BF), torch.randn(N, K, generator=g, device=DEV).mul_(K ** -0.5).to(BF)
    b, r = torch.randn(N, generator=g, device=DEV), torch.randn(T, N, generator=g, device=DEV).to(BF)
    zr, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    for bias, res, keep, out in [(b, r, True, BF), (None, None, False, BF), (b, None, True, torch.float32),
                                 (None, r, False, torch.float32), (None, None, False, torch.float32)]:
        pre = zr + b.double() if bias is not None else zr
        zbuf, z = _inside((T, N), BF, 7.0) if keep else (None, None)
        buf, view = _inside((T, N), out, 7.0)
        moe.linear(x, w, bias, act, res, z, out=view)
        ref = _act64(pre, act) + (r.double() if res is not None else 0)
        # z's own error, times the slope's largest value (1.13 for gelu), and a few roundings of
        # fp32 in the activation: exp is good to |z| 2^-22
        zerr = (K + 2) * 2.0 ** -23 * (size + (b.double().abs() if bias is not None else 0))
        aerr = 1.2 * zerr + (pre.abs() + 8) * 2.0 ** -21 * pre.abs() + 2.0 ** -23 * ref.abs()
        within(view, ref, aerr + HALF[out] * (ref.abs() + aerr), f"y {act}")
        assert _around(buf, 7.0)
        if keep:
            within(z, pre, zerr + HALF[BF] * (pre.abs() + zerr), "z")
            assert _around(zbuf, 7.0)
    apart, into = moe.linear(x, w, b, act, r), r.clone()
    assert torch.equal(moe.linear(x, w, b, act, into, out=into), apart)


def test_refusals_in_one_thread_are_not_another_s():
    """moe_last_error is the calling thread's own."""
    L, said = moe.lib(), {}
    z = torch.zeros(4, 64, dtype=BF, device=DEV)
    refused, fine = threading.Event(), threading.Event()

    def bad():
        assert fine.wait(30)
        with pytest.raises(moe.MoEError, match="overlaps"):
            moe.swiglu(z, out=z.view(-1)[:128].view(4, 32))
        said["bad"] = L.moe_last_error().decode()
        refused.set()

    def good():
        moe.swiglu(z)
        fine.set()
        assert refused.wait(30)
        said["good"] = L.moe_last_error().decode()

    threads = [threading.Thread(target=f) for f in (bad, good)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert "overlaps" in said["bad"] and said["good"] == ""


@pytest.mark.parametrize("T,N", [(1 << 29, 136), (1 << 30, 64)])
def test_more_tiles_than_a_grid_row(T, N):
    """2^23 and more blocks of 256 threads: more than a launch may have along one axis."""
    K, chunk = 8, 1 << 20
    say(f"linear {T} {N} {K}")
    torch.cuda.empty_cache()
    w = torch.randn(N, K, device=DEV).to(BF)
    x = torch.randn(chunk, K, device=DEV).to(BF).repeat(T // chunk, 1)  # the rows repeat, so the results do
    y = torch.empty(T, N, dtype=BF, device=DEV)
    y.fill_(float("nan"))
    moe.linear(x, w, out=y)
    a, b = x[:chunk].double(), w.double().t()
    ref, size = a @ b, a.abs() @ b.abs()
    within(y[:chunk], ref, product_bound(ref, size, K, BF), "y")
    for i in range(chunk, T, chunk):
        assert torch.equal(y[i:i + chunk], y[:chunk]), i
    del x, y
    torch.cuda.empty_cache()

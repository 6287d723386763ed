"""The AdamW step against its formula in 64 bits; 8-bit moments against the formula in plain fp32 arithmetic, bit for bit.

Bounds, u = 2^-24 (one rounding of fp32). m: both factors' and both products' roundings, clipping, and the sum:
5 u (|b1 m| + |(1-b1) g|). v: the same with one product more: 6 u v'. The step w = rate m' / (sqrt(v') root + eps): the
relative error of the denominator is half v's (3 u), sqrt, root's rounding, product, sum (4 u); division, rate, product (4 u);
and m's own: 11 u |w| + 5 u rate (|b1 m| + |(1-b1) g|) / denominator, doubled for products of these errors. p keep: 2 u |p|;
the difference: u |p'|. A bf16 parameter rounds once more: 2^-8 |p'|.
"""
import math

import numpy as np
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, gen, say, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
SIZES = [1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 40007]
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def make(sizes, param, grad, bits, master, seed, used=True):
    """State with moments of earlier steps (or of none), gradients, on the CPU."""
    g = gen(seed)
    params = [(torch.randn(n, generator=g) * 0.05).to(param) for n in sizes]
    grads = [(torch.randn(n, generator=g) * 10.0 ** float(torch.randint(-4, 1, (1,), generator=g))).to(grad) for n in sizes]
    s = moe.AdamWState.zeros(params, bits, master)
    if used:
        for i, n in enumerate(sizes):
            a, e = s.starts()[i], s.starts()[i + 1]
            m, r = torch.zeros(e - a), torch.zeros(e - a)
            m[:n] = torch.randn(n, generator=g) * 1e-2
            r[:n] = torch.rand(n, generator=g) * 1e-2
            if bits == 32:
                s.m[a:e], s.v[a:e] = m, r * r
            else:
                for x, codes, scale in ((m, s.m, s.m_scale), (r, s.v, s.v_scale)):
                    c, sc = encode(x)
                    codes[a:e], scale[a // 128:e // 128] = c, sc
            if s.master is not None:
                s.master[a:a + n] += torch.randn(n, generator=g) * 1e-4
    return s, grads


def to_gpu(s, grads):
    def up(t):
        return None if t is None else t.to(DEV)
    return moe.AdamWState([up(p) for p in s.params], up(s.m), up(s.v), up(s.m_scale), up(s.v_scale), up(s.master)), [up(g) for g in grads]


def encode(x):
    """Codes and scales of whole blocks, in fp32. numpy's quotients and roots are rounded correctly; torch's
    root on the CPU is one unit off for one value in 160."""
    x = x.numpy().reshape(-1, 128)
    most = np.maximum(np.abs(x).max(axis=1), np.float32(2.0 ** -100))
    inv = np.float32(448) * (np.float32(1) / most)
    c = np.clip(x * inv[:, None], np.float32(-448), np.float32(448))
    return torch.from_numpy(c).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), torch.from_numpy(most / np.float32(448))


def check(before, grads, after, step, clip=1.0, what="", lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1):
    """`after` (from the GPU) is `before` (CPU) one step on."""
    b1, b2 = betas
    fix1, fix2 = 1 - b1 ** step, 1 - b2 ** step
    eight = before.m.dtype == torch.uint8
    for i, p0 in enumerate(before.params):
        n, a, e = p0.numel(), before.starts()[i], before.starts()[i + 1]
        g = grads[i]
        if g is None:
            continue
        m0, v0 = before.moments(i)
        old = before.master[a:a + n] if before.master is not None and p0.dtype == BF else p0.reshape(-1)
        m0, v0, p0d, gd = (t.double().reshape(-1) for t in (m0, v0, old, g))
        gd = gd * clip
        m, v = b1 * m0 + (1 - b1) * gd, b2 * v0 + (1 - b2) * gd * gd
        size = b1 * m0.abs() + (1 - b1) * gd.abs()
        den = torch.sqrt(v / fix2) + eps
        w = lr / fix1 * m / den
        p = p0d * (1 - lr * weight_decay) - w
        err = 2 * (11 * U * w.abs() + 5 * U * lr / fix1 * size / den) + 2 * U * p0d.abs() + U * p.abs()
        got = after.params[i].reshape(-1)
        if before.master is not None and p0.dtype == BF:
            within(after.master[a:a + n], p, err, f"{what} master {i}")
            assert torch.equal(got.cpu(), after.master[a:a + n].cpu().to(BF)), f"{what} parameter {i} is not its copy rounded"
            assert not after.master[a + n:e].any()
        else:
            within(got, p, err + (HALF[BF] * (p.abs() + err) if p0.dtype == BF else 0.0), f"{what} parameter {i}")
        if eight:
            # products and sums rounded one by one in fp32
            gf = g.reshape(-1).float() * torch.tensor(clip, dtype=F32)
            mf, vf = before.moments(i)
            mf = mf.reshape(-1) * b1 + gf * (1.0 - b1)
            vf = vf.reshape(-1) * b2 + (gf * gf) * (1.0 - b2)
            for x, codes, scale, name in ((mf, after.m, after.m_scale, "m"), (torch.from_numpy(np.sqrt(vf.numpy())), after.v, after.v_scale, "v")):
                c, sc = encode(torch.nn.functional.pad(x, (0, e - a - n)))
                assert torch.equal(scale[a // 128:e // 128].cpu(), sc), f"{what} scales of {name} {i}"
                assert torch.equal(codes[a:e].cpu(), c), f"{what} codes of {name} {i}"
        else:
            within(after.m[a:a + n], m, 5 * U * size, f"{what} m {i}")
            within(after.v[a:a + n], v, 6 * U * v, f"{what} v {i}")
            assert not after.m[a + n:e].any() and not after.v[a + n:e].any()


def down(s):
    def cpu(t):
        return None if t is None else t.cpu().clone()
    return moe.AdamWState([p.cpu().clone() for p in s.params], cpu(s.m), cpu(s.v), cpu(s.m_scale), cpu(s.v_scale), cpu(s.master))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF, BF, True), (BF, F32, True), (BF, BF, False), (F32, BF, False)])
@pytest.mark.parametrize("step", [1, 1000])
def test_a_step(param, grad, master, bits, step):
    say(f"adamw {param} {grad} master={master} bits={bits} step={step}")
    s, grads = make(SIZES, param, grad, bits, master, step + bits, used=step > 1)
    d, dg = to_gpu(s, grads)
    moe.adamw(d, dg, step, **HYPER)
    check(s, grads, d, step, what=f"step {step}", **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_one_after_another(bits):
    s, _ = make(SIZES, BF, BF, bits, True, 5, used=False)
    d, _ = to_gpu(s, [])
    for step in range(1, 6):
        grads = [(torch.randn(n, generator=gen(step * 100 + i)) * 0.1).to(BF) for i, n in enumerate(SIZES)]
        before = down(d)
        moe.adamw(d, [g.to(DEV) for g in grads], step, **HYPER)
        check(before, grads, d, step, what=f"step {step}", **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_and_types_mixed(bits):
    """130 tensors: three launches; both types of parameters and gradients, shapes, one without a gradient, empty ones."""
    g = gen(3)
    params, grads = [], []
    for i in range(130):
        n = [0, 1, 3, 130, 2049, 777, 64][i % 7]
        shape = (n // 64, 64) if n and n % 64 == 0 else (n,)
        params.append((torch.randn(shape, generator=g) * 0.1).to(BF if i % 3 else F32))
        grads.append(None if i == 17 else torch.randn(shape, generator=g).to(BF if i % 2 else F32))
    s = moe.AdamWState.zeros(params, bits)
    d, _ = to_gpu(s, [])
    d.params[17].fill_(3.0)
    moe.adamw(d, [None if t is None else t.to(DEV) for t in grads], 1, **HYPER)
    check(s, grads, d, 1, what="mixed", **HYPER)
    assert bool((d.params[17] == 3.0).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [(BF, BF), (F32, F32), (BF, F32)])
def test_parameters_and_gradients_off_16_bytes(param, grad, bits):
    """Views that start at any value of a larger buffer, and what lies around them."""
    g = gen(9)
    n = 3001
    for shift in (0, 1, 3, 8, 13):
        buf = torch.randn(n + 40, generator=g).to(param)
        gb = torch.randn(n + 40, generator=g).to(grad)
        db, dgb = buf.to(DEV), gb.to(DEV)
        before = moe.AdamWState.zeros([buf[shift:shift + n]], bits)
        d = moe.AdamWState.zeros([db[shift:shift + n]], bits)
        moe.adamw(d, [dgb[shift + 1:shift + 1 + n]], 1, **HYPER)
        check(before, [gb[shift + 1:shift + 1 + n]], d, 1, what=f"shift {shift}", **HYPER)
        assert torch.equal(db[:shift].cpu(), buf[:shift]) and torch.equal(db[shift + n:].cpu(), buf[shift + n:])
        assert torch.equal(dgb.cpu(), gb)


@pytest.mark.parametrize("bits", [32, 8])
def test_rates_on_the_device(bits):
    for step, lr, clip in ((1, 1e-2, 0.25), (7, 3e-4, 1.0), (100000, 1e-3, 0.0)):
        s, grads = make([300, 5000], BF, F32, bits, True, step)
        d, dg = to_gpu(s, grads)
        lr32 = torch.tensor([lr], device=DEV)
        moe.adamw(d, dg, torch.tensor([step], dtype=torch.int32, device=DEV), lr32, betas=(0.9, 0.999), eps=1e-6, weight_decay=0.0,
                  grad_scale=torch.tensor([clip], device=DEV))
        check(s, grads, d, step, clip, "device", lr=float(lr32.item()), betas=(0.9, 0.999), eps=1e-6, weight_decay=0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas,eps,decay", [((0.0, 0.0), 1e-8, 0.0), ((0.0, 0.999), 1e-3, 0.5), ((0.95, 0.0), 1.0, 0.0)])
def test_rates_at_their_ends(betas, eps, decay, bits):
    s, grads = make([1000], F32, F32, bits, False, 11)
    d, dg = to_gpu(s, grads)
    hyper = dict(lr=0.5, betas=betas, eps=eps, weight_decay=decay)
    moe.adamw(d, dg, 3, **hyper)
    check(s, grads, d, 3, what=str(betas), **hyper)


def test_zero_gradients_and_tiny_ones():
    """Blocks of zeros keep code and moment 0; magnitudes below the least scale are finite."""
    p = torch.ones(512)
    for scale in (0.0, 1e-30, 1e-38, 1e-18):
        grads = [torch.randn(512, generator=gen(1)) * scale]
        s = moe.AdamWState.zeros([p], 8)
        d = moe.AdamWState.zeros([p.to(DEV)], 8)
        moe.adamw(d, [grads[0].to(DEV)], 1, **HYPER)
        check(s, grads, d, 1, what=f"{scale}", **HYPER)
        assert bool(torch.isfinite(d.params[0]).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite_stay_where_they_are(bits):
    s, grads = make([1000], F32, F32, bits, False, 4)
    grads[0][5] = float("nan")
    grads[0][700] = float("inf")
    d, dg = to_gpu(s, grads)
    moe.adamw(d, dg, 2, **HYPER)
    bad = ~torch.isfinite(d.params[0].cpu())
    assert bad.nonzero().flatten().tolist() == [5, 700]
    m, v = (t.cpu() for t in d.moments(0))
    blocks = {0, 5} if bits == 8 else set()
    for t in (m, v):
        off = (~torch.isfinite(t)).nonzero().flatten().tolist()
        assert 5 in off and 700 in off
        # an infinity takes the scale of its block of 128, a NaN only its own code
        assert all(i in (5, 700) or (bits == 8 and i // 128 == 5) for i in off), (off, blocks)


def test_captured_steps():
    """A captured step replayed: step number, rate and gradients are read anew each time."""
    for bits in (32, 8):
        s, grads = make([4000, 33], BF, BF, bits, True, 8)
        d, dg = to_gpu(s, grads)
        step = torch.tensor([1], dtype=torch.int32, device=DEV)
        lr = torch.tensor([1e-3], device=DEV)
        clip = torch.tensor([1.0], device=DEV)
        twin = moe.AdamWState([p.clone() for p in d.params], d.m.clone(), d.v.clone(), *(None if t is None else t.clone() for t in (d.m_scale, d.v_scale, d.master)))
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                moe.adamw(d, dg, step, lr, grad_scale=clip)
        for k in range(1, 5):
            step.fill_(k)
            lr.fill_(1e-3 * k)
            clip.fill_(1.0 / k)
            for g in dg:
                g.mul_(0.5)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            moe.adamw(twin, dg, step, lr, grad_scale=clip)
            torch.cuda.synchronize()
            for a, b in zip(d.params + [d.m, d.v, d.master], twin.params + [twin.m, twin.v, twin.master]):
                assert torch.equal(a, b), f"replay {k}"


def test_streams_and_the_same_bits():
    s, grads = make([100000, 17], BF, BF, 8, True, 21)
    runs = []
    for k in range(3):
        d, dg = to_gpu(s, grads)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            moe.adamw(d, dg, 2, **HYPER)
        torch.cuda.synchronize()
        runs.append(d)
    check(s, grads, runs[0], 2, what="stream", **HYPER)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r.params + [r.m, r.v, r.master], runs[0].params + [runs[0].m, runs[0].v, runs[0].master]))


def test_elements_past_32_bits():
    """A tensor of more than 2^31 elements: its first, middle and last parts."""
    n = (1 << 31) + 1000
    say(f"n = {n}")
    p = torch.full((n,), 0.5, dtype=BF, device=DEV)
    g = torch.full((n,), 0.25, dtype=BF, device=DEV)
    for a in (0, n // 2, n - 3000):
        g[a:a + 3000] = torch.randn(3000, generator=gen(a % 97)).to(BF).to(DEV)
    d = moe.AdamWState.zeros([p], 8, master=False)
    moe.adamw(d, [g], 1, **HYPER)
    torch.cuda.synchronize()
    for a in (0, n // 2 // 128 * 128, (n - 3000) // 128 * 128 + 128):
        k = min(2560, n - a)
        part = moe.AdamWState.zeros([torch.full((k,), 0.5, dtype=BF)], 8, master=False)
        end = a + (k + 127) // 128 * 128
        after = moe.AdamWState([p[a:a + k]], d.m[a:end], d.v[a:end], d.m_scale[a // 128:end // 128], d.v_scale[a // 128:end // 128])
        check(part, [g[a:a + k].cpu()], after, 1, what=f"from {a}", **HYPER)


def test_binding_refusals_on_the_gpu():
    p, g = torch.zeros(256, device=DEV), torch.zeros(256, device=DEV)
    s = moe.AdamWState.zeros([p])
    for bad in ([g[:128]], [g.double()], [g.cpu()], [torch.zeros(256, 2, device=DEV)[:, 0]]):
        with pytest.raises(ValueError):
            moe.adamw(s, bad, 1, 1e-3)
    with pytest.raises(moe.MoEError):
        moe.adamw(moe.AdamWState.zeros([p, p]), [g, g], 1, 1e-3)  # named twice
    with pytest.raises(moe.MoEError):
        moe.adamw(s, [p], 1, 1e-3)
    with pytest.raises(moe.MoEError):
        moe.adamw(s, [g], 0, 1e-3)
    with pytest.raises(ValueError):
        moe.adamw(moe.AdamWState([p], s.m[:128], s.v), [g], 1, 1e-3)
    with pytest.raises(TypeError):
        moe.adamw(s, [g], torch.ones(1, device=DEV), 1e-3)
    assert not p.any() and math.isfinite(p.sum().item())

"""8-bit moments on the GPU: over thousands of steps beside moments in 32 bits, and every code, scale and fine byte against the
formula in plain fp32 arithmetic. The bounds of the long runs are derived in test_adamw_moments_cpu.py."""
import numpy as np
import pytest
import torch

import moe_ffn_int4_amd as moe
from adamw_formula import Moments
from train_util import DEV, gen, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _pair(sizes, dtype=F32):
    def params():
        return [torch.zeros(n, dtype=dtype, device=DEV) for n in sizes]
    return moe.AdamWState.zeros(params(), 8), moe.AdamWState.zeros(params(), 32)


def _ratio(eight, wide, i):
    return torch.sqrt(eight.moments(i)[1] / wide.moments(i)[1])


def _follows(ratio, what):
    mean, far = ratio.mean().item(), ((ratio - 1).abs() > 0.38).float().mean().item()
    say(f"{what}: mean {mean:.4f} deviation {ratio.std().item():.4f}")
    assert abs(mean - 1) <= 0.02 and far <= 0.01, (what, mean, far)


@pytest.mark.parametrize("beta2", [0.99, 0.999])
@pytest.mark.parametrize("scene", ["fall", "rise", "one"])
def test_second_moments_over_a_long_run(beta2, scene):
    """Gradients of half of the elements fall or rise; or one of a block falls, and the others stay as they are."""
    say(f"{scene} beta2={beta2}")
    n = 8200
    eight, wide = _pair([n])
    g0 = torch.Generator(device=DEV).manual_seed(3)
    some = torch.arange(n, device=DEV) % (128 if scene == "one" else 2) == 0
    warm = int(3 / (1 - beta2))
    for t in range(3 * warm):
        late = t >= warm
        g = torch.randn(n, device=DEV, generator=g0)
        factor = {"fall": 0.1 if late else 1.0, "rise": 1.0 if late else 0.25, "one": 1.0 if late else 20.0}[scene]
        g = torch.where(some, g * factor, g)
        for s in (eight, wide):
            moe.adamw(s, [g], t + 1, 1e-3, betas=(0.9, beta2))
    _follows(_ratio(eight, wide, 0)[~some if scene == "one" else some], f"{scene} {beta2}")


def test_default_betas_at_rest_and_the_parameters():
    """Several tensors, bf16 gradients: v, and how far the parameters of both states are apart."""
    sizes = [5, 129, 3000, 9001]
    eight, wide = _pair(sizes)
    g0 = torch.Generator(device=DEV).manual_seed(4)
    for t in range(3000):
        grads = [torch.randn(n, device=DEV, generator=g0).to(BF) for n in sizes]
        for s in (eight, wide):
            moe.adamw(s, grads, t + 1, 1e-3)
    for i in (2, 3):
        _follows(_ratio(eight, wide, i), f"tensor {i}")
        d = (eight.params[i] - wide.params[i]).norm() / wide.params[i].norm()
        # each step is off by what sqrt(v) is, 0.066 of it at most (one deviation), and m's 0.010
        assert d.item() <= 0.1, d


def test_a_first_moment_turns_its_sign():
    n = 4096
    eight, wide = _pair([n])
    g = torch.randn(n, generator=gen(5)).to(DEV)
    turned = g.clone()
    turned[1::2] *= -1
    for t in range(800):
        for s in (eight, wide):
            moe.adamw(s, [g if t < 300 else turned], t + 1, 1e-3, betas=(0.99, 0.999))
    m8, m32 = (s.moments(0)[0][1::2] for s in (eight, wide))
    least = g.abs().reshape(-1, 128).amax(1).repeat_interleave(128)[1::2] * 2.0 ** -6 / 448
    assert ((m8 - m32).abs() <= 4 * 0.032 * torch.maximum(m32.abs(), least)).all()


def test_a_captured_step_whose_number_stands_still():
    n = 8192
    eight, wide = _pair([n])
    g = torch.randn(n, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for s in (eight, wide):
                moe.adamw(s, [g], 1000, 1e-3, betas=(0.9, 0.99))
    torch.cuda.synchronize()
    g0 = torch.Generator(device=DEV).manual_seed(6)
    for t in range(900):
        g.normal_(generator=g0)
        if t >= 300:
            g[::2] *= 0.1
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    _follows(_ratio(eight, wide, 0)[::2], "captured")


# ------------------------------------------------------------------ bit for bit

def _same(state, i, want, what):
    a, e = state.starts()[i], state.starts()[i + 1]
    fine = torch.zeros(e - a) if state.fine is None else state.fine[a:e]
    for got, ref, name in ((state.m[a:e], want.m, "m"), (state.v[a:e], want.v, "v"), (fine, want.fine, "fine"),
                           (state.m_scale[a // 128:e // 128], want.m_scale, "m_scale"), (state.v_scale[a // 128:e // 128], want.v_scale, "v_scale")):
        assert np.array_equal(got.cpu().numpy(), ref), f"{what}: {name}"


@pytest.mark.parametrize("device", [False, True])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.95), (0.99, 0.0)])
def test_codes_and_what_they_leave(betas, device):
    """Six steps of gradients of all magnitudes, one of them zeros; the step's number from the host or the device, small and large."""
    sizes = [1, 127, 128, 129, 2049, 40007]
    state = moe.AdamWState.zeros([torch.zeros(n, dtype=BF, device=DEV) for n in sizes], 8)
    want = [Moments(n) for n in sizes]
    for t, number in enumerate((1, 2, 3, 77, 100000, 2 ** 31 - 1)):
        r = np.random.default_rng(100 * t + len(betas))
        grads = [(r.standard_normal(n) * np.exp(r.uniform(-18, 3, n)) * (t != 3)).astype(np.float32) for n in sizes]
        moe.adamw(state, [torch.from_numpy(g).to(DEV) for g in grads],
                  torch.tensor([number], dtype=torch.int32, device=DEV) if device else number, 1e-3, betas=betas)
        for i, (w, g) in enumerate(zip(want, grads)):
            w.step(g, number, betas)
            _same(state, i, w, f"step {number} tensor {i}")
    assert any(w.fine.any() for w in want) or betas[0] == 0.0


@pytest.mark.parametrize("alone", [False, True])
def test_a_state_that_is_made_of_tensors(alone):
    """With fine bytes behind v's codes, and of codes alone; a gradient that is None leaves all of it."""
    sizes = [300, 4000]
    r = np.random.default_rng(7)
    plane = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (4480, 4480 if alone else 8960)]
    state = moe.AdamWState([torch.zeros(n, device=DEV) for n in sizes], *plane, *(torch.zeros(35, device=DEV) for _ in range(2)))
    want = [Moments(n, not alone) for n in sizes]
    for t in range(4):
        grads = [r.standard_normal(n).astype(np.float32) for n in sizes]
        moe.adamw(state, [None if t == 2 else torch.from_numpy(grads[0]).to(DEV), torch.from_numpy(grads[1]).to(DEV)], t + 1, 1e-3, betas=(0.9, 0.95))
        for i, (w, g) in enumerate(zip(want, grads)):
            if i or t != 2:
                w.step(g, t + 1, (0.9, 0.95))
            _same(state, i, w, f"step {t} tensor {i}")
    zero = [None, torch.zeros(4000, device=DEV)]
    for n in (4096, 0):
        with pytest.raises(ValueError):
            moe.adamw(moe.AdamWState(state.params, state.m, state.v[:n], state.m_scale, state.v_scale), zero, 1, 1e-3, betas=(0.9, 0.95))
    if alone:
        for betas in ((0.9, 0.999), (0.95, 0.95)):
            with pytest.raises(moe.MoEError):
                moe.adamw(state, zero, 1, 1e-3, betas=betas)
        with pytest.raises(moe.MoEError):
            moe.adamw(state, zero, 1, 1e-3)  # the default betas


@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_whose_square_is_infinite(bits):
    """v of its element (8 bits: of its block) is infinite, the step 0 but for the decay; other blocks and a clipped gradient are as ever."""
    g = torch.ones(512, device=DEV)
    g[130] = 1e20
    for clip, hit in ((1.0, True), (1e-10, False)):
        s = moe.AdamWState.zeros([torch.ones(512, device=DEV)], bits)
        moe.adamw(s, [g], 1, 0.5, weight_decay=0.0, grad_scale=torch.tensor([clip], device=DEV))
        p = s.params[0]
        # a first step is lr g / (|g| + eps)
        assert bool(torch.isfinite(p).all()) and abs(p[0].item() - (1 - 0.5 * clip / (clip + 1e-8))) <= 1e-6 and (p[130].item() == 1.0) == hit
        m, v = s.moments(0)
        bad = (~torch.isfinite(v)).nonzero().flatten().tolist()
        assert bad == ([] if not hit else [130] if bits == 32 else list(range(128, 256))), bad
        assert bool(torch.isfinite(m).all())


def test_past_32_bits():
    """What the hash takes of an element's place past 2^32, and the fine bytes there."""
    n = (1 << 32) + 300
    say(f"n = {n}")
    p = torch.zeros(n, dtype=BF, device=DEV)
    g = torch.zeros(n, dtype=BF, device=DEV)
    first, last = slice(0, 256), slice(1 << 32, n)
    for s in (first, last):
        g[s] = torch.randn(s.stop - s.start, generator=gen(8)).to(BF).to(DEV)
    state = moe.AdamWState.zeros([p], 8, master=False)
    moe.adamw(state, [g], 1, 1e-3)
    moe.adamw(state, [g], 2, 1e-3)
    torch.cuda.synchronize()
    for s in (first, last):
        w = Moments(s.stop - s.start)
        w.start = s.start
        for t in (1, 2):
            w.step(g[s].float().cpu().numpy(), t, (0.9, 0.999))
        e = slice(s.start, s.start + w.m.size)
        for got, ref, name in ((state.m[e], w.m, "m"), (state.v[e], w.v, "v"), (state.fine[e], w.fine, "fine")):
            assert np.array_equal(got.cpu().numpy(), ref), f"{name} from {s.start}"
    assert not state.fine[256:1 << 20].any() and not state.m[256:1 << 20].any()

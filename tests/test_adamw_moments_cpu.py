"""8-bit moments over a long run, in the formula that the GPU tests hold the kernel to; where a state keeps what its codes leave.

Bounds of the long runs. What is kept stands in steps of q <= 1/8/14 = 0.0089 of the value. A step changes sqrt(v) by about
(1 - b2) |g^2 / v - 1| / 2 of it, 0.49 (1 - b2) on average for normal gradients, and the block's scale by as much again; a
rounding up or down by its nearness has a variance of at most q times the change, and a deviation decays by 1 - b2 a step: at rest the variance
of sqrt(v) is at most q (2 * 0.49 (1 - b2)) / (2 (1 - b2)) = 0.0044, its standard deviation at most 0.066 of it. After gradients fall to a
tenth, deviations of a larger value are still on their way (sqrt(v) falls by up to (1 - b2) / 2 a step, so twice the variance): 0.094. Of 2048 elements the mean then is within
0.094 / 45 * 4 = 0.9 % of 1 and, for the curvature of the square, half the variance, 0.45 %; 2 % is allowed, and four deviations, 38 %, for 99 elements of 100.
m: a rounding has at most a quarter of q^2, a deviation decays by 1 - b1: at most q / 2 / sqrt(1 - b1^2), 0.010, 0.014 and 0.032 of m for b1 =
0.9, 0.95 and 0.99; four of these for every element. Where a gradient ends, m_t = b1^t m_0 decays as fast as the deviations do: those of T
steps, of variance (q m_t)^2 / 4 each, become sum_t b1^(2 (T - t)) (q b1^t m_0)^2 / 4 = T (q m_T)^2 / 4, so 0.5 q sqrt(T) of m_T with T = 10 / (1 - b1):
0.045, 0.063 and 0.141.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

import moe_ffn_int4_amd as moe
from adamw_formula import BLOCK, F, Moments, decode, dither, encode, low

INVALID = 1
BASE = 0x10000000000


def follow_v(beta2, scene, keep, after=2, seed=1, n=4096):
    """sqrt(v) in 8 bits over sqrt(v) in 64, `after` times 3 / (1 - beta2) steps after a change, of the elements whose gradients changed (`one`: of the others)."""
    r = np.random.default_rng(seed)
    half, one = np.arange(n) % 2 == 0, np.arange(n) % BLOCK == 0
    s, v = Moments(n, keep), np.zeros(n)
    warm = int(3 / (1 - beta2))
    for t in range((1 + after) * warm):
        late = t >= warm
        g = r.standard_normal(n)
        if scene == "fall" and late:
            g[half] *= 0.1
        elif scene == "rise" and not late:
            g[half] *= 0.25
        elif scene == "one" and not late:
            g[one] *= 20.0
        g = g.astype(F)
        s.step(g, t + 1, (0.9, beta2))
        v = beta2 * v + (1 - beta2) * g.astype(np.float64) ** 2
    ratio = s.values()[1] / np.sqrt(v)
    return ratio[~one if scene == "one" else half]


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
@pytest.mark.parametrize("scene", ["rest", "fall", "rise", "one"])
def test_second_moments_follow(beta2, scene):
    ratio = follow_v(beta2, scene, True)
    assert abs(ratio.mean() - 1) <= 0.02, ratio.mean()
    assert np.mean(np.abs(ratio - 1) <= 0.38) >= 0.99, np.percentile(ratio, [1, 50, 99])


def test_codes_alone_do_not_follow():
    """What the fine bits are for: without them sqrt(v) stands still."""
    assert follow_v(0.99, "fall", False).mean() > 5 and follow_v(0.999, "rise", False).mean() < 0.6


@pytest.mark.parametrize("scene", ["rest", "fall", "rise", "one"])
def test_codes_alone_at_their_largest_betas(scene):
    """What is documented of them at beta2 = 0.95, 240 steps after a change."""
    ratio = follow_v(0.95, scene, False, 4)
    low, high = np.percentile(ratio, [1, 99])
    assert 0.8 <= low and high <= 1.5, (low, high)


@pytest.mark.parametrize("beta1,bound", [(0.9, 0.010), (0.95, 0.014), (0.99, 0.032)])
@pytest.mark.parametrize("then", [0.0, -1.0, 1.4])
def test_first_moments_follow(beta1, bound, then):
    """A steady gradient that ends, turns its sign, or grows."""
    g = np.random.default_rng(2).standard_normal(4096).astype(F)
    s, m = Moments(4096), np.zeros(4096)
    warm = int(10 / (1 - beta1))
    for t in range(2 * warm):
        now = g * F(then if t >= warm else 1.0)
        # half of each block goes on, so that its scale stays
        now[::2] = g[::2]
        s.step(now, t + 1, (beta1, 0.95))
        m = beta1 * m + (1 - beta1) * now.astype(np.float64)
    got = s.values()[0][1::2]
    # values of less than 2^-6 / 448 of the block's largest have its step: q of that instead of q of themselves
    least = np.abs(g).reshape(-1, BLOCK).max(axis=1).repeat(BLOCK)[1::2] * 2.0 ** -6 / 448
    err = np.abs(got - m[1::2])
    allowed = 4 * (bound if then else 0.00446 * warm ** 0.5) * np.maximum(np.abs(m[1::2]), least)
    assert (err <= allowed).all(), (err / allowed).max()


def test_a_step_number_that_stands_still():
    r = np.random.default_rng(4)
    s, v = Moments(4096), np.zeros(4096)
    for t in range(900):
        g = (r.standard_normal(4096) * (0.1 if t >= 300 else 1.0)).astype(F)
        s.step(g, 1000, (0.9, 0.99))
        v = 0.99 * v + 0.01 * g.astype(np.float64) ** 2
    ratio = s.values()[1] / np.sqrt(v)
    assert abs(ratio.mean() - 1) <= 0.02 and np.mean(np.abs(ratio - 1) <= 0.38) >= 0.99


def test_what_codes_leave():
    """The kept digits: nearest below or above, zero for zeros, and both ends of a code's half step."""
    r = np.random.default_rng(5)
    x = (r.standard_normal(128 * 64) * np.exp(r.uniform(-12, 0, 128 * 64))).astype(F)
    x[5], x[200] = 0.0, -0.0
    for random in (np.zeros(x.size, np.uint32), np.full(x.size, 0xFFFF, np.uint32), dither(np.arange(x.size), 3, x) & np.uint32(0xFFFF)):
        codes, scales, k = encode(x, random)
        assert k.min() >= -7 and k.max() <= 7 and k[5] == k[200] == 0
        value = decode(codes, scales, np.zeros_like(k)).astype(np.float64)
        assert np.array_equal(decode(codes, scales, k)[k == 0], value[k == 0].astype(F))
        step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(value / scales.repeat(128)), 1e-30))), 2.0 ** -6) / 8 * scales.repeat(128)
        # within a fourteenth of a code's step, and the roundings of fp32
        assert (np.abs(decode(codes, scales, k) - x) <= step / 14 * 1.0001 + 4 * 2.0 ** -24 * np.abs(x)).all()
    # codes 448 and 416 with what lies half way: the ends of the half step
    edge = np.zeros(128, F)
    edge[:3] = 448, 432, -432
    codes, scales, k = encode(edge, np.full(128, 0xFFFF, np.uint32))
    assert list(k[:3]) == [0, 7, -7] or list(np.abs(k[:3])) == [0, 7, 7]


def test_dither_is_uniform():
    """Over elements, steps and moments, each of 64 bins within six deviations of its share."""
    n = 1 << 18
    zeros = np.zeros(n, F)
    sets = [dither(np.arange(n), 7, zeros), dither(np.arange(n) + (1 << 33), 7, zeros), dither(np.arange(n) * 8, 3, zeros),
            np.array([dither(np.array([9]), t, zeros[:1])[0] for t in range(1 << 14)], np.uint32),
            dither(np.full(n, 5), 2, np.random.default_rng(0).standard_normal(n).astype(F))]
    for x in sets:
        for part in (x & np.uint32(0xFFFF), x >> np.uint32(16)):
            h, _ = np.histogram(part, 64, (0, 65536))
            share = x.size / 64
            assert (np.abs(h - share) <= 6 * share ** 0.5).all()
    assert not np.array_equal(sets[0], sets[1])


def test_where_a_state_keeps_them():
    p = [torch.zeros(130), torch.zeros(7)]
    s = moe.AdamWState.zeros(p, 8)
    assert s.m.shape == (384,) and s.v.shape == (768,) and s.fine.shape == (384,) and s.fine.data_ptr() == s.v.data_ptr() + 384
    alone = moe.AdamWState(p, s.m, s.v[:384], s.m_scale, s.v_scale)
    assert alone.fine is None and [t.shape for t in alone.moments(0)] == [(130,), (130,)]
    again = moe.AdamWState(p, s.m, torch.cat([alone.v, torch.zeros_like(alone.v)]), s.m_scale, s.v_scale)
    assert not again.fine.any() and all(torch.equal(x, y) for i in (0, 1) for x, y in zip(again.moments(i), alone.moments(i)))
    wide = moe.AdamWState.zeros(p, 32)
    assert wide.fine is None and wide.v.shape == (384,)


def test_moments_are_codes_and_what_is_kept():
    r = np.random.default_rng(6)
    state = moe.AdamWState.zeros([torch.zeros(300)], 8)
    s = Moments(300)
    for t in range(3):
        s.step((r.standard_normal(300) * 10.0 ** -t).astype(F), t + 1, (0.9, 0.99))
    for name in ("m", "m_scale", "v_scale"):
        getattr(state, name).copy_(torch.from_numpy(getattr(s, name)))
    state.v[:384], state.v[384:] = torch.from_numpy(s.v), torch.from_numpy(s.fine)
    assert s.fine.any()
    m, v = state.moments(0)
    want_m, root = s.values()
    assert np.array_equal(m.numpy(), want_m[:300]) and np.array_equal(v.numpy(), (root * root)[:300])
    assert low(np.array([0x0F, 0x07, 0x09, 0x08], np.uint8)).tolist() == [-1, 7, -7, -8]


# ------------------------------------------------- refusals of the C entry point

@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from moe_ffn_int4_amd import build
        build.build()
    return moe.lib()


def at(i):
    return BASE + i * (1 << 44)


def call(L, bits=8, fine=1 << 20, betas=(0.9, 0.99), **kw):
    t = dict(param=at(0), grad=at(1), master=at(2), m=at(3), v=at(4), m_scale=at(5), v_scale=at(6), n=1000, types=0)
    t.update(kw)
    if bits == 32:
        t["m_scale"] = t["v_scale"] = 0
    h = moe._AdamWHyper(1e-3, *betas, 1e-8, 0.1, 1, None, None, None, fine)
    return L.moe_adamw((ctypes.c_uint64 * 9)(*t.values()), 1, ctypes.byref(h), bits, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(fine=0), "beta2 = 0.99"), (dict(fine=0, betas=(0.91, 0.95)), "beta1 = 0.91"), (dict(fine=0, betas=(0.0, 0.951)), "codes alone"), (dict(fine=24), "fine = 24"), (dict(fine=-8), "fine = -8"), (dict(bits=32), "with bits 32"),
    # over v's own codes, before and behind; over another buffer
    (dict(fine=1008), "overlaps"), (dict(fine=-1008), "overlaps"), (dict(fine=at(3) - at(4)), "overlaps"), (dict(fine=at(0) + 1984 - at(4)), "overlaps"),
    (dict(fine=at(1) - at(4) - 1008), "overlaps"),
])
def test_refusals(L, kw, needle):
    assert call(L, **kw) == INVALID
    said = L.moe_last_error().decode()
    assert needle in said, said


def test_allowed(L):
    """Right behind or before the codes; the call then ends at the device, past the checks."""
    for fine in (1024, -1024, 1 << 20):
        assert call(L, fine=fine) != INVALID, L.moe_last_error()
    assert call(L, bits=32, fine=0, betas=(0.99, 0.999)) != INVALID
    assert call(L, fine=0, betas=(0.9, 0.95)) != INVALID

"""Activations and slopes at every bf16 value, in fp32, against 64 bits and the header's bound."""
import math

import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TINY = 2.0 ** -119


def _values():
    """Every finite bf16 value."""
    v = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(BF)
    return v[torch.isfinite(v)].to(DEV)


def _exponent(z, act):
    c = math.sqrt(8 / math.pi)
    return {"silu": z, "gelu": z * z / 2, "gelu_tanh": c * (z + 0.044715 * z ** 3)}[act]


def _phi(z):
    # by erfc: ndtr is 0 from z = -8.375 on here, where Phi is exp(-35.07) / (8.375 sqrt(2 pi)) = 2.8e-17
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def _value(z, act):
    return z * (_phi(z) if act == "gelu" else torch.sigmoid(_exponent(z, act)))


def _slope(z, act):
    """The slope's two terms; past +-90 its limit."""
    c = z.clamp(-90, 90)
    if act == "gelu":
        return _phi(z), c * torch.exp(-c * c / 2) / math.sqrt(2 * math.pi)
    s, t = torch.sigmoid(_exponent(z, act)), torch.sigmoid(-_exponent(z, act))
    inner = 1.0 if act == "silu" else math.sqrt(8 / math.pi) * (1 + 0.134145 * c * c)
    return s, c * s * t * inner


def _bound(size, z, act):
    # the exponent matters where the exponential does; past +-120 it is 0 or infinite
    e = _exponent(z, act).abs().clamp(max=120.0)
    return (2.0 ** -19 + e * 2.0 ** -21) * size + TINY


def _inside(got, ref, bound, z, what):
    over = (got.double() - ref).abs() - bound
    at = int(over.argmax())
    assert bool(torch.isfinite(got).all()), what
    assert over[at].item() <= 0, f"{what}: {got[at].item()} for {ref[at].item()} at z = {z[at].item()}"


@pytest.mark.parametrize("rows", [1, 65536])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(act, rows):
    """x W^T gives z itself: one value a row and a unit weight, or one row and each value a weight."""
    say(f"{act} {rows}")
    v = _values()
    v = v[v.abs() < 1e37]  # whose products with 0 and sums with themselves are exact
    n = v.numel() // 8 * 8
    v, x, w = v[:n], torch.zeros(n if rows > 1 else 1, 8, dtype=BF, device=DEV), torch.zeros(8 if rows > 1 else n, 8, dtype=BF, device=DEV)
    x[:, 0] = v if rows > 1 else 1.0
    w[:, 0] = 1.0 if rows > 1 else v
    y = moe.linear(x, w, act=act, out_dtype=torch.float32)
    z = v.double()
    ref = _value(z, act)
    for col in (0, 7) if rows > 1 else (None,):
        _inside(y[0] if col is None else y[:, col], ref, _bound(ref.abs(), z, act), z, act)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes(act):
    """dy = 1 in a single row: db is the slope in fp32."""
    say(act)
    v = _values()
    v = v[:v.numel() // 8 * 8].view(1, -1).contiguous()
    dz, db = moe.linear_dz(torch.ones_like(v), v, act)
    z = v[0].double()
    a, b = _slope(z, act)
    bound = _bound(torch.maximum(a.abs(), b.abs()), z, act)
    _inside(db, a + b, bound, z, act)
    _inside(dz[0], a + b, bound + HALF[BF] * ((a + b).abs() + bound), z, act)


def test_swiglu():
    v = _values()
    v = v[v.abs() < 1e37]
    v = v[:v.numel() // 8 * 8].view(1, -1).contiguous()
    z = torch.cat([v, torch.ones_like(v)], 1)
    g = v[0].double()
    ref = _value(g, "silu")
    bound = _bound(ref.abs(), g, "silu")
    _inside(moe.swiglu(z)[0], ref, bound + HALF[BF] * (ref.abs() + bound), g, "swiglu")
    a, b = _slope(g, "silu")
    slope = _bound(torch.maximum(a.abs(), b.abs()), g, "silu")
    dz = moe.swiglu_backward(torch.ones_like(v), z)[0]
    _inside(dz[:v.numel()], a + b, slope + HALF[BF] * ((a + b).abs() + slope), g, "swiglu's g")
    _inside(dz[v.numel():], ref, bound + HALF[BF] * (ref.abs() + bound), g, "swiglu's u")

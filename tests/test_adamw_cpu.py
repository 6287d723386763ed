"""Refusals of the AdamW step, before any HIP call."""
import ctypes
import os

import pytest
import torch

import moe_ffn_int4_amd as moe

OK, INVALID = 0, 1
F = 0x10000000000  # aligned addresses, far apart, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from moe_ffn_int4_amd import build
        build.build()
    return moe.lib()


def at(i):
    return F + i * (1 << 44)


def tensor(i=0, **kw):
    """The words of a moe_adamw_tensor of 1000 bf16 values with 32-bit moments."""
    t = dict(param=at(10 * i), grad=at(10 * i + 1), master=at(10 * i + 2), m=at(10 * i + 3), v=at(10 * i + 4),
             m_scale=0, v_scale=0, n=1000, types=0)
    t.update(kw)
    return list(t.values())


EIGHT = dict(m_scale=at(5), v_scale=at(6))


def call(L, tensors, bits=32, count=None, **kw):
    words = sum(tensors, [])
    h = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1, step_device=None, lr_device=None, grad_scale=None)
    h.update(kw)
    arr = (ctypes.c_uint64 * max(len(words), 1))(*[w & (2 ** 64 - 1) for w in words])
    return L.moe_adamw(arr, len(tensors) if count is None else count, ctypes.byref(moe._AdamWHyper(*h.values())), bits, None)


def said(L):
    return L.moe_last_error().decode()


@pytest.mark.parametrize("kw,needle", [
    (dict(bits=16), "bits = 16"), (dict(count=-1), "count = -1"), (dict(count=(1 << 20) + 1), "count ="),
    (dict(step=0), "step = 0"), (dict(step=-3), "step = -3"), (dict(lr=-1.0), "lr"), (dict(lr=float("nan")), "lr"),
    (dict(lr=float("inf")), "lr"), (dict(beta1=1.0), "beta1"), (dict(beta1=-0.1), "beta1"), (dict(beta2=1.5), "beta2"),
    (dict(beta2=float("nan")), "beta2"), (dict(eps=-1e-8), "eps"), (dict(weight_decay=float("inf")), "weight_decay"),
    (dict(step_device=F + 2), "step_device"), (dict(lr_device=F + 1), "lr_device"), (dict(grad_scale=F + 2), "grad_scale"),
])
def test_call_refusals(L, kw, needle):
    assert call(L, [tensor()], **kw) == INVALID
    assert needle in said(L), said(L)


@pytest.mark.parametrize("bits,kw,needle", [
    (32, dict(n=-1), "n = -1"), (32, dict(n=(1 << 34) + 1), "n ="), (32, dict(param=0), "param is NULL"),
    (32, dict(grad=0), "grad is NULL"), (32, dict(m=0), "m is NULL"), (32, dict(v=0), "v is NULL"),
    (32, dict(param=at(0) + 1), "param"), (32, dict(param=at(0) + 2, types=1), "param"), (32, dict(grad=at(1) + 2, types=1 << 32), "grad"),
    (32, dict(master=at(2) + 4), "master"), (32, dict(m=at(3) + 8), "m is not"), (32, dict(v=at(4) + 4), "v is not"),
    (32, EIGHT, "bits 32"), (32, dict(v_scale=at(6)), "bits 32"),
    (8, dict(), "m_scale is NULL"), (8, dict(m_scale=at(5)), "v_scale is NULL"), (8, dict(EIGHT, m_scale=at(5) + 2), "m_scale"),
    # what is written overlaps: itself, its gradient, the end of the last block of codes
    (32, dict(grad=at(0)), "overlaps"), (32, dict(grad=at(0) + 1998), "overlaps"), (32, dict(master=at(3) + 16), "overlaps"),
    (32, dict(v=at(3) + 3984), "overlaps"), (32, dict(grad=at(4) + 3998), "overlaps"),
    (8, dict(EIGHT, v=at(3) + 1008), "overlaps"), (8, dict(EIGHT, v_scale=at(5) + 28), "overlaps"),
])
def test_tensor_refusals(L, bits, kw, needle):
    assert call(L, [tensor(1, **({} if bits == 32 else dict(m_scale=at(15), v_scale=at(16)))), tensor(**kw)], bits) == INVALID
    assert needle in said(L), said(L)


def test_a_tensor_named_twice(L):
    assert call(L, [tensor(0), tensor(1), tensor(0, grad=at(31), master=at(32), m=at(33), v=at(34))]) == INVALID
    assert "param of tensor" in said(L)
    assert call(L, [tensor(0), tensor(1, m=at(3))]) == INVALID
    # one gradient for two tensors is nothing that is written
    assert call(L, [tensor(0), tensor(1, grad=at(1))]) != INVALID
    # a gradient that spans what another tensor writes
    assert call(L, [tensor(0, grad=at(10) - 64), tensor(1)]) == INVALID
    assert "grad of tensor 0" in said(L)
    # neighbours without a gap, in any order
    assert call(L, [tensor(0, m=at(3) + 4000), tensor(1, m=at(3))]) != INVALID


def test_together_too_many(L):
    n = (1 << 34) // 4
    assert call(L, [tensor(i, n=n + 1, master=0) for i in range(4)]) == INVALID
    assert "together" in said(L)


def test_null_arguments(L):
    h = moe._AdamWHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert L.moe_adamw(None, 1, ctypes.byref(h), 32, None) == INVALID
    assert L.moe_adamw(None, 0, None, 32, None) == INVALID


def test_nothing_to_do(L):
    h = moe._AdamWHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert L.moe_adamw(None, 0, ctypes.byref(h), 32, None) == OK
    assert call(L, [tensor(n=0, param=0, grad=0, m=0, v=0)]) == OK


def test_device_rates_are_not_the_hosts(L):
    # lr and step of the host are not read where the device has them; without a GPU the call then ends at the device
    assert call(L, [tensor()], lr=-1.0, lr_device=at(50)) != INVALID
    assert call(L, [tensor()], step=0, step_device=at(50)) != INVALID


def test_state_layout():
    p = [torch.zeros(3, 5, dtype=torch.bfloat16), torch.zeros(129), torch.zeros(0), torch.zeros(128)]
    s = moe.AdamWState.zeros(p, 8)
    assert s.starts() == [0, 128, 384, 384, 512]
    assert s.m.dtype == torch.uint8 and s.m.shape == (512,) and s.m_scale.shape == (4,) and s.master.shape == (512,)
    assert moe.AdamWState.zeros(p[1:], 32).master is None
    assert [t.shape for t in s.moments(0)] == [(3, 5), (3, 5)]
    with pytest.raises(ValueError):
        moe.AdamWState.zeros(p, 16)
    with pytest.raises(ValueError):
        moe.AdamWState.zeros([], 32)


def test_binding_refusals():
    s = moe.AdamWState.zeros([torch.zeros(8)])
    with pytest.raises(ValueError):
        moe.adamw(s, [], 1, 1e-3)
    with pytest.raises(ValueError):
        moe.adamw(s, [torch.zeros(8)], 1, 1e-3)  # not on a GPU


@pytest.mark.parametrize("name", ["step_device", "lr_device", "grad_scale"])
def test_numbers_that_the_step_would_overwrite(L, name):
    for where in (at(0) + 1996, at(2) + 4, at(3), at(4) + 3996):
        assert call(L, [tensor()], **{name: where}) == INVALID
        assert name in said(L) and "of tensor 0" in said(L), said(L)
    # a number may lie in a gradient, which is read alone, or right behind what is written
    assert call(L, [tensor()], **{name: at(1)}) != INVALID
    assert call(L, [tensor()], **{name: at(3) + 4000}) != INVALID

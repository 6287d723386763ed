"""The training operators on tensors of more than 2^31 values: what lies past the 32-bit offsets."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, HALF, U32, product_bound, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(*shape, scale=1.0):
    t = torch.empty(*shape, dtype=BF, device=DEV).normal_()
    return t.mul_(scale) if scale != 1.0 else t


def _product(got, a, b, red, what):
    ref, size = a.double() @ b.double(), a.double().abs() @ b.double().abs()
    within(got, ref, product_bound(ref, size, red, BF), what)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_weights_past_32_bits(rows):
    """The last of 40 experts starts past 2^31 values; it and the first alone have rows."""
    E, N, K = 40, 16384, 4096
    say(f"{rows} rows, {E * N * K} weights")
    w = _rand(E, N, K, scale=0.1)
    counts = [rows] + [0] * (E - 2) + [rows]
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    x, dy = _rand(2 * rows, K), _rand(2 * rows, N)
    y, dx = moe.grouped_matmul(x, w, off), moe.grouped_matmul_dx(dy, w, off)
    for e, s in ((0, slice(0, rows)), (E - 1, slice(rows, 2 * rows))):
        _product(y[s, -1000:], x[s], w[e, -1000:].t(), K, "y")
        _product(dx[s, -1000:], dy[s], w[e, :, -1000:], N, "dx")
    del w
    dw = moe.grouped_matmul_dw(dy, x, off)
    for e, s in ((0, slice(0, rows)), (E - 1, slice(rows, 2 * rows))):
        _product(dw[e, -1000:], dy[s, -1000:].t(), x[s], rows, "dw")
    assert bool((dw[1] == 0).all()) and bool((dw[E - 2] == 0).all())


@pytest.mark.parametrize("T,N,K", [(70000, 32768, 64), (140000, 16384, 520)])
def test_rows_past_32_bits(T, N, K):
    say(f"linear {T} {N} {K}")
    x, w, r = _rand(T, K), _rand(N, K, scale=0.1), _rand(T, N)
    y = moe.linear(x, w, residual=r)
    dx = moe.linear_dx(y, w)
    tail = slice(T - 300, T)
    ref, size = x[tail].double() @ w.double().t() + r[tail].double(), x[tail].double().abs() @ w.double().abs().t()
    err = (K + 2) * U32 * (size + r[tail].double().abs())
    within(y[tail], ref, err + HALF[BF] * (ref.abs() + err), "y")
    _product(dx[tail], y[tail], w, N, "dx")
    dz, db = moe.linear_dz(y, r, "relu")
    want = torch.where(r[tail].float() > 0, y[tail], torch.zeros_like(y[tail]))
    assert torch.equal(dz[tail], want)
    del x, w, y, dx
    total, size = torch.zeros(N, dtype=torch.float64, device=DEV), torch.zeros(N, dtype=torch.float64, device=DEV)
    for i in range(0, T, 10000):
        total += dz[i:i + 10000].double().sum(0)
        size += dz[i:i + 10000].double().abs().sum(0)
    within(db, total, (T + 1) * U32 * size, "db")


def test_expert_rows_past_32_bits():
    T, k, d = 1 << 15, 8, 8264
    say(f"combine of {T * k * d} values")
    perm = torch.randperm(T * k, device=DEV).to(torch.int32)
    inv = torch.empty_like(perm)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    x, gates = _rand(T, d), torch.rand(T, k, device=DEV)
    xp = moe.permute_rows(x, perm, k)
    for s in (slice(0, 500), slice(T * k - 500, T * k)):
        assert torch.equal(xp[s], x[(perm[s] // k).long()])
    y = moe.combine(xp, inv, gates)
    d_o, dg = moe.combine_backward(x, xp, inv.view(T, k), gates)
    for s in (slice(0, 200), slice(T - 200, T)):
        # every row of a token's pairs is the token's own
        terms = x[s].double().unsqueeze(1) * gates[s].double().unsqueeze(2)
        ref, err = terms.sum(1), (k + 1) * U32 * terms.abs().sum(1)
        within(y[s], ref, err + HALF[BF] * (ref.abs() + err), "y")
        within(d_o[inv.view(T, k)[s].long()], terms, (HALF[BF] + U32) * 1.01 * terms.abs(), "d_o")
        dot = (x[s].double() ** 2).sum(1, keepdim=True).expand(-1, k)
        within(dg[s], dot, (d + 1) * U32 * dot, "d_gates")


def test_more_waves_of_pairs_than_a_grid_row():
    T, k, d = (1 << 21) + 3, 8, 264
    say(f"combine_backward of {T * k} pairs of {d}")
    dy, gates = _rand(T, d), torch.rand(T, k, device=DEV)
    inv = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    o = _rand(T * k, d)
    d_o = torch.full((T * k, d), 7.0, dtype=BF, device=DEV)
    _, dg = moe.combine_backward(dy, o, inv, gates, out=d_o)
    for s in (slice(0, 1000), slice(T // 2, T // 2 + 1000), slice(T - 1000, T)):
        want = (gates[s].unsqueeze(2) * dy[s].float().unsqueeze(1)).to(BF)
        assert torch.equal(d_o.view(T, k, d)[s], want)
        prod = dy[s].double().unsqueeze(1) * o.view(T, k, d)[s].double()
        within(dg[s], prod.sum(2), (d + 1) * U32 * prod.abs().sum(2), "d_gates")

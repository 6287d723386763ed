"""The operators in the order a training step uses them: the layer's forward and backward,
against the same layer in 64 bits, against differences of its loss, and against moe.forward."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, bf16, gen, say

pytestmark = pytest.mark.gpu
# A value passes at most five roundings to bf16 in sequence on its way (up-projection,
# SwiGLU, down-projection, shared sum, output; backward alike), each off by at most half a
# step, 2^-8 relative: 5 * 2^-8 = 2e-2, taken of the norm of the whole tensor.
TOL = 2e-2


def _layer(T, d, E, h, k, seed):
    g = gen(seed)
    p = dict(x=bf16(g, T, d), wr=torch.randn(E, d, generator=g) * 0.05, w13=bf16(g, E, 2 * h, d, scale=d ** -0.5),
             w2=bf16(g, E, d, h, scale=h ** -0.5), s1=bf16(g, h, d, scale=d ** -0.5), s3=bf16(g, h, d, scale=d ** -0.5),
             s2=bf16(g, d, h, scale=h ** -0.5), b1=torch.randn(h, generator=g) * 0.1, dy=bf16(g, T, d))
    return p


def _step(p, k):
    """Forward and backward with the package's operators: y and every gradient."""
    x = p["x"]
    r = moe.route(x, p["wr"], None, k)
    off, perm, inv, gates = r["offsets"], r["perm"], r["inv"], r["gates"]
    T, h = x.shape[0], p["s1"].shape[0]
    # routed experts
    xp = moe.permute_rows(x, perm, k)
    z13 = moe.grouped_matmul(xp, p["w13"], off)
    hid = moe.swiglu(z13)
    o = moe.grouped_matmul(hid, p["w2"], off)
    # shared expert, each projection a dense layer: silu(x s1^T + b1) * (x s3^T)
    z1 = torch.empty(T, h, dtype=torch.bfloat16, device=x.device)
    a1 = moe.linear(x, p["s1"], p["b1"], "silu", z=z1)
    a3 = moe.linear(x, p["s3"])
    hs = a1 * a3
    shared = moe.linear(hs, p["s2"], residual=x)  # with the layer's residual
    y = moe.combine(o, inv, gates, residual=shared)
    # backward
    dy = p["dy"]
    d_o, d_gates = moe.combine_backward(dy, o, inv, gates)
    dw2 = moe.grouped_matmul_dw(d_o, hid, off)
    d_hid = moe.grouped_matmul_dx(d_o, p["w2"], off)
    d_z13 = moe.swiglu_backward(d_hid, z13, out=z13)
    dw13 = moe.grouped_matmul_dw(d_z13, xp, off)
    d_xp = moe.grouped_matmul_dx(d_z13, p["w13"], off)
    ds2 = moe.linear_dw(dy, hs)
    d_hs = moe.linear_dx(dy, p["s2"])
    d_z1, db1 = moe.linear_dz(d_hs * a3, z1, "silu")
    d_a3 = d_hs * a1
    ds1, ds3 = moe.linear_dw(d_z1, x), moe.linear_dw(d_a3, x, out_dtype=torch.float32)
    dx = moe.linear_dx(d_z1, p["s1"], out_dtype=torch.float32)
    dx += moe.linear_dx(d_a3, p["s3"], out_dtype=torch.float32)
    dx += moe.combine(d_xp, inv, top_k=k, residual=dy).float()
    return dict(y=y, x=dx, w13=dw13, w2=dw2, s1=ds1, s3=ds3, s2=ds2, b1=db1, gates=d_gates), r


def _loss64(q, ids, gates, k, dy):
    """sum(y * dy) of the layer in 64 bits with the given routing."""
    x = q["x"]
    T, d = x.shape
    h = q["s1"].shape[0]
    act = torch.nn.functional.silu
    y = x + (act(x @ q["s1"].t() + q["b1"]) * (x @ q["s3"].t())) @ q["s2"].t()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            z = q["w13"][e] @ x[t]
            y = y.index_add(0, torch.tensor([t]), (gates[t, j] * (q["w2"][e] @ (act(z[:h]) * z[h:]))).unsqueeze(0))
    return (y * dy).sum(), y


def _near(got, ref, what):
    err = (got.double().cpu() - ref).norm().item()
    assert err <= TOL * ref.norm().item(), f"{what}: {err:.3e} of {ref.norm().item():.3e}"


@pytest.mark.parametrize("T,d,E,h,k", [(1, 128, 4, 128, 1), (24, 256, 6, 272, 2), (40, 128, 5, 72, 3)])
def test_training_step(T, d, E, h, k):
    say(f"training step T={T} d={d} E={E} h={h} k={k}")
    p = _layer(T, d, E, h, k, T + d)
    got, r = _step({n: t.to(DEV) for n, t in p.items()}, k)
    ids, gates = r["ids"].cpu(), r["gates"].double().cpu()
    names = ["x", "w13", "w2", "s1", "s3", "s2", "b1"]
    q = {n: p[n].double().requires_grad_(True) for n in names}
    gates.requires_grad_(True)
    loss, y = _loss64(q, ids, gates, k, p["dy"].double())
    grads = torch.autograd.grad(loss, [q[n] for n in names] + [gates])
    _near(got["y"], y.detach(), "y")
    for n, ref in zip(names + ["gates"], grads):
        _near(got[n], ref, f"gradient of {n}")
    # differences of the loss along a random direction of each input
    with torch.no_grad():
        for i, n in enumerate(names + ["gates"]):
            base = gates if n == "gates" else q[n]
            v = torch.randn(base.shape, generator=gen(i), dtype=torch.float64)
            eps = 1e-5
            side = []
            for s in (eps, -eps):
                qq = {**q, **({} if n == "gates" else {n: base + s * v})}
                side.append(_loss64(qq, ids, base + s * v if n == "gates" else gates, k, p["dy"].double())[0].item())
            along = (got[n].double().cpu() * v).sum().item()
            want = (side[0] - side[1]) / (2 * eps)
            size = got[n].double().norm().item() * v.norm().item()
            assert abs(along - want) <= TOL * size, f"{n}: {along} along the direction, {want} by differences"


def test_forward_agrees_with_the_fused_layer():
    """The same experts through moe.forward (bf16 experts, tiled) and through the operators."""
    T, d, E, h, k = 200, 256, 5, 384, 2
    p = _layer(T, d, E, h, k, 3)
    p["b1"].zero_()
    c = {n: t.to(DEV) for n, t in p.items()}
    got, _ = _step(c, k)
    ex = moe.Bf16Experts.empty(E, d, h, DEV)
    for e in range(E):
        ex.set_expert(e, c["w13"][e, :h].contiguous(), c["w13"][e, h:].contiguous(), c["w2"][e].contiguous())
    y = moe.forward(c["x"], c["wr"], None, ex, moe.pack_shared(c["s1"], c["s3"], c["s2"]), k)
    _near(got["y"], y.double().cpu() + p["x"].double(), "y")

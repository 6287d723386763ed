"""The operators in the order a program uses them: a layer's gated experts forward and backward, a step of their weights,
and the stepped weights quantized to 4 bits and served token by token."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from test_gpu_adamw import check, down
from train_util import DEV, bf16, gen, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
# A value passes at most five roundings to bf16 in sequence (projections, their product, expert output, sum of the tokens'; backward
# alike), each off by at most 2^-8 relative, taken of the norm of the whole tensor.
TOL = 5 * 2.0 ** -8


def _near(got, ref, what, tol=TOL):
    err = (got.double().cpu() - ref).norm().item()
    assert err <= tol * ref.norm().item(), f"{what}: {err:.3e} of {ref.norm().item():.3e}"


def _layer64(x, w13, w2, off, perm, gates, k):
    """The routed experts' sum for each token, in 64 bits, with the given routing."""
    h = w2.shape[2]
    rows = []
    xp = x[perm.long() // k]
    for e in range(w13.shape[0]):
        z = xp[off[e]:off[e + 1]] @ w13[e].t()
        rows.append((z[:, :h] * torch.sigmoid(z[:, :h]) * z[:, h:]) @ w2[e].t())
    o = torch.cat(rows)
    return torch.zeros_like(x).index_add(0, perm.long() // k, o * gates.reshape(-1)[perm.long()].unsqueeze(1))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("T,d,E,h,k", [(24, 128, 4, 256, 2), (150, 256, 5, 128, 1)])
def test_train_step_quantize_serve(T, d, E, h, k, bits):
    say(f"train and serve T={T} d={d} E={E} h={h} k={k} bits={bits}")
    g = gen(T + bits)
    x, dy, wr = bf16(g, T, d), bf16(g, T, d), (torch.randn(E, d, generator=g) * 0.05)
    w13, w2 = bf16(g, E, 2 * h, d, scale=d ** -0.5), bf16(g, E, d, h, scale=h ** -0.5)
    xd, dyd, wrd = x.to(DEV), dy.to(DEV), wr.to(DEV)
    state = moe.AdamWState.zeros([w13.to(DEV), w2.to(DEV)], bits)
    for step in (1, 2):
        p13, p2 = state.params
        r = moe.route(xd, wrd, None, k)
        off, perm, inv, gates = r["offsets"], r["perm"], r["inv"], r["gates"]
        xp = moe.permute_rows(xd, perm, k)
        z = torch.empty(T * k, 2 * h, dtype=BF, device=DEV)
        o = moe.grouped_matmul(moe.grouped_gated(xp, p13, off, z=z), p2, off)
        y = moe.combine(o, inv, gates)
        d_o, _ = moe.combine_backward(dyd, o, inv, gates)
        hid = torch.empty(T * k, h, dtype=BF, device=DEV)
        dz = moe.grouped_gated_dz(d_o, p2, z, off, y=hid, out=z)
        grads = [moe.grouped_matmul_dw(dz, xp, off, out_dtype=torch.float32), moe.grouped_matmul_dw(d_o, hid, off)]
        dx = moe.combine(moe.grouped_matmul_dx(dz, p13, off), inv, top_k=k)
        q = [t.detach().double().cpu().requires_grad_(True) for t in (x, p13, p2)]
        y64 = _layer64(*q, off.cpu(), perm.cpu(), gates.double().cpu(), k)
        _near(y, y64.detach(), "y")
        for got, ref, n in zip([dx] + grads, torch.autograd.grad((y64 * dy.double()).sum(), q), ("x", "w13", "w2")):
            _near(got, ref, f"gradient of {n}")
        before = down(state)
        moe.adamw(state, grads, step, **HYPER)
        check(before, [t.cpu() for t in grads], state, step, what=f"step {step}", **HYPER)

    # the 32-bit copies in 4 bits; both projections of the layer, for all tokens at once and one by one
    starts, copies = state.starts(), []
    for i, (rows, cols) in enumerate(((2 * h, d), (d, h))):
        copies.append(state.master[starts[i]:starts[i] + E * rows * cols].reshape(E, rows, cols))
    for group in moe.GROUPS:
        (q13, s13), (q2, s2) = ([torch.stack(t) for t in zip(*(moe.quantize_int4(w[e], tiled=True, group=group) for e in range(E)))] for w in copies)
        wide = []
        for w in copies:
            codes, scales = moe.quantize_int4(w, group=group)
            wide.append((moe.unpack_int4(codes).double() * scales.double().repeat_interleave(group, dim=2)).cpu())
        xp = moe.permute_rows(xd, perm, k)
        hid = moe.swiglu(moe.grouped_matmul_int4(xp, q13, s13, off))
        y = moe.combine(moe.grouped_matmul_int4(hid, q2, s2, off), inv, gates, residual=xd)
        ref = _layer64(x.double(), *wide, off.cpu(), perm.cpu(), gates.double().cpu(), k) + x.double()
        _near(y, ref, f"served in groups of {group}")
        t, e = 3, int(r["ids"][3, 0])
        one = moe.linear_int4(moe.swiglu(moe.linear_int4(xd[t:t + 1], q13[e], s13[e])), q2[e], s2[e], out_dtype=torch.float32)
        z = x[t].double() @ wide[0][e].t()
        _near(one[0], (z[:h] * torch.sigmoid(z[:h]) * z[h:]) @ wide[1][e].t(), f"one token, groups of {group}")

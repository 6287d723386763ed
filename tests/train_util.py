"""Plain 64-bit forms and error bounds for the tests of the training operators.

Bounds are elementwise and derived: bf16 products are exact in fp32, and each of
the R additions of a reduction is off by at most one unit in the last place of a partial
sum (2^-23; a matrix unit need not round to nearest), so a sum is off by at most
R 2^-23 sum|a b|. A rounding to bf16 adds half a step, 2^-8 relative to the value.
"""
import torch

U32 = 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DEV = "cuda:0"


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def within(got, ref, bound, what=""):
    """|got - ref| <= bound elementwise, NaN and infinities in the same places."""
    got, ref, bound = got.double().cpu(), ref.double().cpu(), bound.double().cpu()
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} against {tuple(ref.shape)}"
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities"
    if not bool(fine.any()):
        return
    over = ((got - ref).abs() - bound)[fine]
    worst = over.max().item()
    if worst > 0:
        at = (over > 0).sum().item()
        raise AssertionError(f"{what}: {at} of {over.numel()} values past their bound, by up to {worst:.3e}")


def product_bound(ref, abs_sum, red, dtype):
    """Bound of a reduction of length `red` rounded to `dtype`."""
    err = (red + 1) * U32 * abs_sum
    return err + HALF[dtype] * (ref.abs() + err)


def split_counts(P, E, seed, skew=0.0, empty=()):
    """E group sizes that sum to P; the groups in `empty` get none."""
    share = (torch.arange(E, dtype=torch.float64) + 1) ** -skew
    for e in empty:
        share[e] = 0
    if P == 0:
        return [0] * E
    ids = torch.multinomial(share[torch.randperm(E, generator=gen(seed))] if not empty else share, P, True,
                            generator=gen(seed + 1))
    return torch.bincount(ids, minlength=E).tolist()


def offsets_of(counts, start=0):
    o = [start]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32)

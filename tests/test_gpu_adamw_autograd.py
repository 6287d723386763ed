"""Parameters that a step has written, in torch's autograd."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_that_needs_the_old_values(bits):
    """A backward pass through a graph kept over the step raises, as after torch's own optimizers."""
    w = torch.ones(64, 64, device=DEV, requires_grad=True)
    x = torch.ones(2, 64, device=DEV, requires_grad=True)
    state = moe.AdamWState.zeros([w], bits)
    y = (x @ w).sum()
    y.backward(retain_graph=True)
    moe.adamw(state, [w.grad], 1, 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    # a new graph of the stepped weights has their gradient
    w.grad = None
    (x @ w).sum().backward()
    assert bool((w.grad == 2.0).all())


def test_only_what_is_stepped():
    a, b = torch.ones(8, device=DEV), torch.ones(8, dtype=torch.bfloat16, device=DEV)
    with torch.inference_mode():
        c = torch.ones(8, device=DEV)  # keeps no version
    g = torch.ones(8, device=DEV)
    state = moe.AdamWState.zeros([a, b, c])
    before = a._version, b._version, g._version
    moe.adamw(state, [g, None, g], 1, 1e-3)
    assert (a._version, b._version, g._version) == (before[0] + 1, before[1], before[2])
    # a call that is refused steps nothing
    with pytest.raises(moe.MoEError):
        moe.adamw(state, [g, None, g], 0, 1e-3)
    moe.adamw(state, [None, None, None], 1, 1e-3)
    assert a._version == before[0] + 1
    # a view's step is its base's
    base = torch.ones(64, device=DEV)
    was = base._version
    moe.adamw(moe.AdamWState.zeros([base[16:32]]), [torch.ones(16, device=DEV)], 1, 1e-3)
    assert base._version == was + 1 and bool((base[32:] == 1).all())

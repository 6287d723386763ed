"""The product kernels at sizes that the rule sends to each of them, against 64-bit products."""
import pytest
import torch

import moe_ffn_int4_amd as moe
from train_util import DEV, product_bound, say, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("T,N", [(1 << 29, 136), (1 << 30, 64)])
def test_more_tiles_than_a_grid_row(T, N):
    """2^23 and more blocks of 256 threads: more than a launch may have along one axis."""
    K, chunk = 8, 1 << 20
    say(f"linear {T} {N} {K}")
    torch.cuda.empty_cache()
    w = torch.randn(N, K, device=DEV).to(BF)
    x = torch.randn(chunk, K, device=DEV).to(BF).repeat(T // chunk, 1)  # the rows repeat, so the results do
    y = torch.empty(T, N, dtype=BF, device=DEV)
    y.fill_(float("nan"))
    moe.linear(x, w, out=y)
    a, b = x[:chunk].double(), w.double().t()
    ref, size = a @ b, a.abs() @ b.abs()
    within(y[:chunk], ref, product_bound(ref, size, K, BF), "y")
    for i in range(chunk, T, chunk):
        assert torch.equal(y[i:i + chunk], y[:chunk]), i
    del x, y
    torch.cuda.empty_cache()

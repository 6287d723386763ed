"""4-bit products in fp32 where codes are small and an activation is not: the error goes by sum |x scale|, not by sum |x scale code|.

Bound as in test_gpu_int4_product.py, of group sums of x (code + 24) and of 24 x.
"""
import pytest
import torch

import moe_ffn_int4_amd as moe
from test_gpu_int4_product import _product
from train_util import DEV, HALF, offsets_of, say, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _small_codes(g, N, K, group, zero):
    """Codes -1, 0, 1, and 0 in column `zero`, packed and tiled, with scales of one magnitude."""
    codes = torch.randint(-1, 2, (N, K), generator=g, device=DEV)
    codes[:, zero] = 0
    low, high = codes[:, 0::2] & 15, codes[:, 1::2] & 15
    q = (low | high << 4).to(torch.uint8)
    s = 0.01 * (1 + torch.rand(N, K // group, generator=g, device=DEV))
    return *moe.tile_int4(q, s, group), codes.double(), s.double()


@pytest.mark.parametrize("group", [128, 64, 32])
@pytest.mark.parametrize("T,N,K", [(1, 64, 1024), (1, 8192, 1280), (5, 208, 1152), (37, 1024, 2048), (70, 480, 128), (300, 7232, 256), (500, 8336, 512)])
@pytest.mark.parametrize("large", [1.0, 300.0, 2.0 ** 40])
def test_an_outlier_under_a_zero_code(T, N, K, group, large):
    say(f"T={T} N={N} K={K} group={group} large={large}")
    g = torch.Generator(device=DEV).manual_seed(T + N)
    zero = K - 37
    q, s, codes, scales = _small_codes(g, N, K, group, zero)
    x = torch.randn(T, K, generator=g, device=DEV)
    x[:, zero] = large
    x = x.to(BF)
    ref, err = _product(x.double(), codes, scales, group)
    assert ref.abs().max() < 100  # the outlier takes no part in the result
    got = moe.linear_int4(x, q, s, out_dtype=F32)
    within(got, ref, err + HALF[F32] * (ref.abs() + err), "linear")
    sums = x.double().abs() @ scales.repeat_interleave(group, dim=1).t()
    say(f"  error {((got.double() - ref).norm() / ref.norm()).item():.1e} of the result, at most {((got.double() - ref).abs() / sums).max().item() * 2 ** 24:.2f} * 2^-24 of sum |x scale|")
    other = torch.cat([x, x])
    off = offsets_of((T, T))
    got = moe.grouped_matmul_int4(other, torch.stack([q, q]), torch.stack([s, s]), off.to(DEV), out_dtype=F32)
    for half in (got[:T], got[T:]):
        within(half, ref, err + HALF[F32] * (ref.abs() + err), "by expert")
    low = moe.linear_int4(x, q, s)
    within(low, ref, err + HALF[BF] * (ref.abs() + err), "bf16")

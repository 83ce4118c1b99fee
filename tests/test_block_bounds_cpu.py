"""The bounds on whole outputs tell sums in fp32 from sums rounded to the type
on the way (CPU: both planted in a plain product)."""
import pytest
import torch

from block_norms import ONE_ROUNDING, TWO_ROUNDINGS, distance
from block_refs import UNIT


def _product(a, b, dtype, each=None):
    """a @ b with sums in fp32, rounded to the type at the end, or every `each` steps of k too."""
    sum32 = torch.zeros(a.shape[0], b.shape[1])
    for i in range(0, a.shape[1], 32):
        sum32 = sum32 + a[:, i:i + 32].float() @ b[i:i + 32].float()
        if each and i // 32 % (each // 32) == 0:
            sum32 = sum32.to(dtype).float()
    return sum32.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", [128, 3624])
def test_norms_tell_where_sums_were_rounded(k, dtype):
    g = torch.Generator().manual_seed(k)
    exact_dz, w = torch.randn(64, k, generator=g, dtype=torch.float64), torch.randn(k, 256, generator=g).to(dtype)
    dz = exact_dz.to(dtype)
    u = UNIT[dtype]
    assert distance(_product(dz, w, dtype), dz.double() @ w.double()) <= ONE_ROUNDING * u
    assert distance(_product(dz, w, dtype), exact_dz @ w.double()) <= TWO_ROUNDINGS * u
    if k > 1000:
        for each in (32, 256):
            assert distance(_product(dz, w, dtype, each), exact_dz @ w.double()) > TWO_ROUNDINGS * u

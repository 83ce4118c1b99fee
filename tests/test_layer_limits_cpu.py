"""Cross attention's scale: the exponentials are base 2, so it must stay finite
times log2(e) in fp32, or a zero score would become NaN (CPU: every refusal
comes before any GPU call; no rows, so what is not refused does nothing)."""
import ctypes

import pytest

import libutil
import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd import attention as A
from ring_allreduce_reduce_amd import block as B

LARGEST = 3.4028234663852886e38


def call(name, struct, scale):
    libutil.lib()
    a = struct(dtype=3, batch=0, queries=1, keys=1, heads=1, kv_heads=1, head_dim=64, scale=scale)
    return B._fn(name)(ctypes.byref(a), None)


@pytest.mark.parametrize("name, struct", [("ringar_cross_attention", A.ringar_cross_attention_t),
                                          ("ringar_cross_attention_backward", A.ringar_cross_attention_backward_t)])
def test_scale_stays_finite_in_base_2(name, struct):
    # 2.3e38 * log2(e) = 3.318e38 < 3.403e38 < 3.463e38 = 2.4e38 * log2(e)
    assert call(name, struct, 2.3e38) == ra.SUCCESS
    for scale in (2.4e38, LARGEST):
        assert call(name, struct, scale) == ra.INVALID_ARGUMENT

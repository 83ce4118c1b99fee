"""Tensors the block operators refuse before they look at the device (CPU)."""
import pytest
import torch

import libutil
import ring_allreduce_reduce_amd as ra


def test_negated_views_are_refused():
    """Their memory holds the values with the other sign."""
    libutil.lib()
    z = torch.randn(4, 1, dtype=torch.complex64).conj().imag
    assert z.is_neg()
    t, w = torch.zeros(4, 1), torch.zeros(8, 1)
    for call in (lambda: ra.layer_norm(z), lambda: ra.layer_norm(t, out=z), lambda: ra.linear(z, w), lambda: ra.linear(t, w, residual=z),
                 lambda: ra.linear_backward(z, t, w), lambda: ra.layer_norm_backward(t, t, z, t), lambda: ra.gated_ffn(t, z)):
        with pytest.raises(ra.RingarError, match="negated") as e:
            call()
        assert e.value.code == ra.INVALID_ARGUMENT

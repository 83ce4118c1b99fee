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


def test_arguments_that_are_no_tensors_with_a_stream():
    """Refused as they are without a stream."""
    libutil.lib()
    t = torch.zeros(4, 8)

    class Stream:
        device_index = 0

    import ring_allreduce_reduce_amd.block as B
    for call in (lambda s: ra.layer_norm("x", stream=s), lambda s: ra.linear(t, 3, stream=s), lambda s: ra.linear_backward(t, t, t, [1], stream=s)):
        with pytest.raises(ra.RingarError) as e:
            call(None)
        assert e.value.code == ra.INVALID_ARGUMENT
    for bad in ("x", 3, [1]):
        with pytest.raises(ra.RingarError) as e:
            B._On(Stream(), t, None, bad)
        assert e.value.code == ra.INVALID_ARGUMENT


def test_an_activation_that_is_no_name():
    libutil.lib()
    t = torch.zeros(4, 8)
    for act in ([], {}, 3, None):
        with pytest.raises(ra.RingarError) as e:
            ra.linear(t, t, act=act)
        assert e.value.code == ra.INVALID_ARGUMENT and "activation" in str(e.value)

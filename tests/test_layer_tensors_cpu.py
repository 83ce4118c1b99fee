"""Tensors that the root-mean-square norm, dropout and attention refuse before they look at the device (CPU)."""
import pytest
import torch

import libutil
import ring_allreduce_reduce_amd as ra


def test_negated_views_are_refused():
    """Their memory holds the values with the other sign, dropout's offset in memory among them."""
    libutil.lib()
    t, h, one = torch.zeros(4, 8), torch.zeros(1, 2, 2, 8), torch.ones(1, dtype=torch.int64)
    neg = torch._neg_view
    for call in (lambda: ra.dropout(t, 0.5, 1, neg(one)), lambda: ra.dropout_backward(t, 0.5, 1, neg(one)), lambda: ra.dropout(neg(t), 0.5, 1),
                 lambda: ra.dropout(t, 0.5, 1, residual=neg(t)), lambda: ra.rms_norm(t, neg(t[0])), lambda: ra.rms_norm(t, residual=t, sum_out=neg(t)),
                 lambda: ra.rms_norm_backward(t, t, neg(t[:, 0])), lambda: ra.cross_attention(h, neg(h), h),
                 lambda: ra.cross_attention(h, h, h, key_lengths=neg(one.int()))):
        with pytest.raises(ra.RingarError, match="negated") as e:
            call()
        assert e.value.code == ra.INVALID_ARGUMENT

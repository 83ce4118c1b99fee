"""Which operands of the block operators may share memory: every refusal comes
before any GPU call (CPU)."""
import pytest

import ring_allreduce_reduce_amd as ra
from test_block_abi_cpu import P, call, lin, norm


def square(**kw):
    return lin(**{**dict(in_features=64, out_features=64, ldx=64, ldw=64, ldy=64, pre=None), **kw})


@pytest.mark.parametrize("where", range(3))
def test_only_the_residual_may_be_the_output(where):
    """y over x, the weight or the bias, each of which is the residual too."""
    args = square(y=P[where], residual=P[where], ldr=64, bias=P[2])
    assert call("ringar_linear", args) == ra.INVALID_USAGE
    assert "y overlaps " + ("x", "weight", "bias")[where] in ra.ringar_last_error()


@pytest.mark.parametrize("which", ["weight", "bias"])
def test_only_the_norms_input_may_be_its_output(which):
    assert call("ringar_layer_norm", norm(y=P[0], **{which: P[0]})) == ra.INVALID_USAGE
    assert "y overlaps " + which in ra.ringar_last_error()

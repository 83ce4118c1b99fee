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


def test_a_single_row_beside_a_strided_output():
    """A vector, or a matrix of one row, between the rows of a strided output
    shares nothing with it; one that reaches a row of it does."""
    import host_runtime
    import tempfile
    with tempfile.TemporaryDirectory() as folder:
        host_runtime.run(host_runtime.build(folder), """
            es = 2
            for row in (0, 2):
                inside = P[3] + (row * 160 + 64) * es            # y: 64 of every 160 columns
                for change, code in ((dict(bias=inside), 0), (dict(bias=inside + 32 * es), 0), (dict(bias=inside + 33 * es), 2),
                                     (dict(bias=inside - es), 2), (dict(weight=inside, bias=inside), 0)):
                    got = call("ringar_layer_norm", norm(ldy=160, **change))
                    assert got == code, (row, change, got, ra.ringar_last_error())
            # statistics of 4 bytes between the input's rows, whole words apart
            assert call("ringar_layer_norm", norm(ldx=160, mean=P[0] + 64 * es)) == 0
            assert call("ringar_layer_norm", norm(ldx=160, mean=P[0] + 63 * es + 2 - 4)) == 2
            # more rows than one, another stride: refused as before
            assert call("ringar_linear", lin(ldy=160, residual=P[4] + 64 * es, ldr=32)) == 2
        """)

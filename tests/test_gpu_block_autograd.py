"""What the block operators owe autograd: a caller's tensor written through
`out` counts as changed in place."""
import pytest
import torch

import ring_allreduce_reduce_amd as ra

pytestmark = pytest.mark.gpu


def _calls():
    x, w, r = torch.randn(6, 64, device="cuda"), torch.randn(64, 64, device="cuda"), torch.randn(6, 64, device="cuda")
    return {"layer_norm": lambda t: ra.layer_norm(t, out=t), "linear": lambda t: ra.linear(x, w, residual=t, out=t),
            "linear into a view": lambda t: ra.linear(x[:3], w, out=t[3:]), "gated_ffn": lambda t: ra.gated_ffn(x, torch.cat((w, w)), out=t),
            "other stream": lambda t: ra.layer_norm(r, out=t, stream=torch.cuda.current_stream())}


@pytest.mark.parametrize("name", ["layer_norm", "linear", "linear into a view", "gated_ffn", "other stream"])
def test_an_output_written_over_a_saved_tensor_is_noticed(name):
    print("case autograd", name, flush=True)
    call = _calls()[name]
    leaf = torch.randn(6, 64, device="cuda", requires_grad=True)
    t = leaf * 2.0
    loss = (t * t).sum()                     # keeps t
    with torch.no_grad():
        before = t._version
        call(t.detach())
    assert t._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_refused_calls_and_inference_tensors():
    print("case autograd refused", flush=True)
    t = torch.randn(6, 64, device="cuda")
    before = t._version
    with pytest.raises(ra.RingarError):
        ra.linear(t, torch.randn(64, 64, device="cuda"), residual=t, out=t)
    assert t._version == before
    ra.layer_norm(t)
    assert t._version == before
    with torch.inference_mode():
        u = torch.randn(6, 64, device="cuda")
        want = ra.layer_norm(u)
        assert torch.equal(ra.layer_norm(u, out=u), want)
    assert torch.equal(ra.layer_norm(u, out=u), ra.layer_norm(want))

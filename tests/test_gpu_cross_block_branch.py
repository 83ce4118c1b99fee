"""What the tensor-parallel cross-attention layer adds to the residual stream, and
what its backward pass adds to the stream's gradient, on their own: the residual is ten
times as large and would hide them.

Bound: test_gpu_cross_block_example's, of the branch's norm (its roundings are those
counted there), and the rounding of the sum with the residual: half a step of it, and
three more of fp32's for the fp32 form's own sums and differences."""
import pytest
import torch

import layer_refs as L
from ring_allreduce_reduce_amd.examples.tensor_parallel_cross_block import CrossBlock

pytestmark = pytest.mark.gpu
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("ranks,batch,rows,keys,width,heads,kv,d", [(2, 3, 17, 65, 136, 4, 2, 40), (4, 2, 130, 300, 256, 8, 4, 64)])
def test_the_branch_alone(ranks, batch, rows, keys, width, heads, kv, d, dtype):
    print("case", ranks, batch, rows, keys, width, heads, kv, d, dtype, flush=True)
    block = CrossBlock(ranks, width, heads, kv, d, dtype, seed=rows)
    gen = torch.Generator(device="cuda").manual_seed(rows + 1)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dtype)  # noqa: E731
    x, h, dy, states = normal(batch, rows, width), normal(batch, rows, width), normal(batch, rows, width), normal(batch, keys, width)
    lengths = torch.tensor([keys - i * keys // (2 * batch) for i in range(batch)], dtype=torch.int32, device="cuda")
    y, saved = block.forward(x, h, states, lengths, step=3)
    grads = block.backward(dy, saved)
    want, plain = block.plain(x, h, states, lengths, L.kept(batch * rows, width, block.p, block.seed, 3).cuda(), dy)
    terms = width + keys + batch * rows + heads * d + 64
    bound = 42 * UNIT[dtype] if dtype != torch.float32 else 4 * terms * UNIT[dtype]
    s = saved[1]
    for got, stream, ref, ref_stream, times, what in ((y, s, want, x.double() + h.double(), 1, "y"), (grads["x"], dy, plain["x"], dy, 2, "dx")):
        branch = ref.detach().double() - ref_stream.detach().double()
        off = (got.detach().double() - stream.detach().double() - branch).norm()
        allowed = times * bound * branch.norm() + (UNIT[dtype] + 3 * 2.0 ** -24) * got.detach().double().norm()
        print(what, float(off / branch.norm()), float(allowed / branch.norm()), float(branch.norm() / stream.detach().double().norm()), flush=True)
        assert allowed < 0.5 * branch.norm() and off <= allowed, what

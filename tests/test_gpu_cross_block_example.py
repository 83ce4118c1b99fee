"""The tensor-parallel cross-attention layer (norm with residual, projections,
cross attention, AllReduce, dropout with residual, and their backward passes)
against the unsharded layer in fp32.

Bound: every value passes at most 10 roundings to the type in a row (sum, norm,
projections, P or dS, attention's output, partial product, the AllReduce's
hops, dropout; likewise backward), each at most a unit roundoff of what it
rounds; the softmax turns a relative distance r of its scores' operands into
at most 2 r max|score|, max|score| below 8 here, of a part of the output that
is added to the residual, so norms of outputs are off by at most (10 + 2 * 8 *
2) units, of gradients by at most twice that."""
import pytest
import torch

import layer_refs as L
import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd.examples.tensor_parallel_block import distance
from ring_allreduce_reduce_amd.examples.tensor_parallel_cross_block import CrossBlock

pytestmark = pytest.mark.gpu
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("ranks,batch,rows,keys,width,heads,kv,d", [(1, 1, 1, 7, 64, 2, 2, 32), (2, 3, 17, 65, 136, 4, 2, 40), (4, 2, 130, 300, 256, 8, 4, 64)])
def test_tensor_parallel_cross_block(ranks, batch, rows, keys, width, heads, kv, d, dtype):
    print("case", ranks, batch, rows, keys, width, heads, kv, d, dtype, flush=True)
    block = CrossBlock(ranks, width, heads, kv, d, dtype, seed=rows)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dtype)  # noqa: E731
    x, h, dy, states = normal(batch, rows, width), normal(batch, rows, width), normal(batch, rows, width), normal(batch, keys, width)
    lengths = torch.tensor([keys - i * keys // (2 * batch) for i in range(batch)], dtype=torch.int32, device="cuda")
    y, saved = block.forward(x, h, states, lengths, step=5)
    grads = block.backward(dy, saved)
    torch.cuda.synchronize()
    assert ra.ringar_get_async_error(torch.cuda.current_stream().cuda_stream) == ra.SUCCESS
    keep = L.kept(batch * rows, width, block.p, block.seed, 5)
    assert torch.equal(block.mask((batch * rows, width), 5).cpu(), keep)
    want, plain = block.plain(x, h, states, lengths, keep.cuda(), dy)
    # fp32: the sums' own roundings in place of the type's
    terms = width + keys + batch * rows + heads * d + 64
    bound = 42 * UNIT[dtype] if dtype != torch.float32 else 4 * terms * UNIT[dtype]
    assert distance(y, want) <= bound
    for k in plain:
        assert distance(grads[k], plain[k]) <= 2 * bound, k

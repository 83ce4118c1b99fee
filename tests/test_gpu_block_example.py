"""The tensor-parallel block (layer norm, gated feed-forward, linear, their
backward passes and the AllReduce together) against the unsharded block in
fp32.

Bound: every value passes at most 8 roundings to the type in a row (norm,
gated output, partial product, the AllReduce's hops; backward: dy's products,
dz, the hops, the norm), each at most a unit roundoff of what it rounds, and
the block does not amplify relative distances by more than 2 in norm."""
import pytest
import torch

import ring_allreduce_reduce_amd as ra
from ring_allreduce_reduce_amd.examples.tensor_parallel_block import Block, distance

pytestmark = pytest.mark.gpu
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("ranks,rows,width,hidden", [(1, 7, 64, 128), (2, 33, 136, 264), (4, 300, 256, 1024)])
def test_tensor_parallel_block(ranks, rows, width, hidden, dtype):
    print("case", ranks, rows, width, hidden, dtype, flush=True)
    block = Block(ranks, width, hidden, dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    x = torch.randn(rows, width, device="cuda", generator=gen).to(dtype)
    dy = torch.randn(rows, width, device="cuda", generator=gen).to(dtype)
    y, saved = block.forward(x)
    grads = block.backward(dy, saved)
    torch.cuda.synchronize()
    assert ra.ringar_get_async_error(torch.cuda.current_stream().cuda_stream) == ra.SUCCESS
    want, plain = block.plain(x, dy)
    # fp32: the sums' own roundings (hidden terms) in place of the type's
    bound = 16 * UNIT[dtype] if dtype != torch.float32 else 2 * (hidden + rows + 64) * UNIT[dtype]
    assert distance(y, want) <= bound
    for k in plain:
        assert distance(grads[k], plain[k]) <= bound, k

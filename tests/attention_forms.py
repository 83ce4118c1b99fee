"""Sizes that lead attention's forward pass to the kernels of many rows: four
waves of 32 rows that share their tiles, and two such groups of waves that take
the tiles in turn; with one part of the keys and with several."""
import torch

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

# (kernel's waves along the rows, along the keys), parts of the keys?, batch, queries, keys, heads, key heads, head_dim
SIXTEEN = [
    ((4, 1), False, 8, 33, 193, 24, 12, 64),
    ((4, 1), False, 8, 33, 193, 24, 12, 80),
    ((4, 1), False, 8, 33, 193, 24, 12, 128),
    ((4, 1), True, 8, 100, 1100, 10, 5, 80),
    ((4, 2), False, 8, 33, 300, 24, 12, 64),
    ((4, 2), False, 8, 33, 300, 24, 12, 80),
    ((4, 2), False, 8, 33, 300, 24, 12, 128),
    ((4, 2), True, 8, 33, 1100, 24, 12, 80),
    ((4, 2), True, 8, 100, 1500, 10, 5, 128),
]
THIRTY_TWO = [
    ((4, 1), False, 8, 200, 193, 10, 5, 64),
    ((4, 1), False, 8, 33, 193, 24, 12, 80),
    ((4, 1), False, 8, 33, 193, 24, 12, 128),
    ((4, 1), True, 8, 33, 300, 24, 12, 64),
    ((4, 1), True, 8, 33, 449, 12, 6, 80),
    ((4, 1), True, 8, 33, 449, 12, 6, 128),
    ((4, 2), False, 8, 200, 300, 10, 5, 64),
    ((4, 2), True, 8, 100, 700, 10, 5, 64),
]
CASES = [(dtype, *c) for dtype, cases in ((F16, SIXTEEN), (BF16, SIXTEEN), (F32, THIRTY_TWO)) for c in cases]


def tile_keys(dtype):
    """Keys of a tile in these kernels."""
    return 32 if dtype == F32 else 64


def lengths_of(dtype, keys):
    """Eight sequences: all keys, none, one, a tile, one more, an even and an odd number of tiles, all but one."""
    t = tile_keys(dtype)
    return [keys, 0, 1, t, t + 1, 2 * t, 3 * t - 1, keys - 1]

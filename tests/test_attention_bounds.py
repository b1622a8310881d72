"""What the attention tests' limits would let pass, on the oracle's side."""
import math

import pytest
import torch

from test_gpu_attn_long import LIMIT, off


@pytest.mark.parametrize("n", [4000, 9001, 40001])
def test_the_limit_sees_a_tile_left_out(n):
    """The definition without one tile of 128 keys is past the limit, whichever
    tile it is."""
    g = torch.Generator().manual_seed(42)
    q, k, v = (torch.randn(m, 128, generator=g).bfloat16().double() for m in (3, n, n))
    p = torch.exp(1.5 * q @ k.T / math.sqrt(128))
    want = p @ v / p.sum(1, keepdim=True)
    for at in range(0, n, 128):
        x = p.clone()
        x[:, at:at + 128] = 0
        assert off(x @ v / x.sum(1, keepdim=True), want) > LIMIT, at

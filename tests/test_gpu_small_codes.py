"""attn_select over bounds of any power of two that an E8M0 code says, those below 2^-106 included (kv_index writes none)."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import long_ref
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low,high", [(0, 6), (14, 27), (0, 255), (245, 255)])
@pytest.mark.parametrize("nodes,G,D", [(1, 1, 64), (3, 8, 128), (20, 4, 64)])
def test_scores_of_any_code(nodes, G, D, low, high):
    P, Hkv, page, n_sel = 90, 2, 16, 17
    g = torch.Generator().manual_seed(low + nodes)
    # sums that differ in a few bits, so that the codes decide between pages
    codes = torch.randint(1, 4, (P, Hkv, 2, D), generator=g, dtype=torch.int8)
    codes[:, :, 1] -= 4
    exps = torch.randint(low, high, (P, Hkv), generator=g, dtype=torch.uint8)
    q = torch.randn(nodes, Hkv * G, D, generator=g).bfloat16()
    table = torch.randperm(P, generator=g).int()[None]
    index = mx.PageIndex(codes.to(dev()), exps.to(dev()), page)
    cu = torch.tensor([0, nodes], dtype=torch.int32, device=dev())
    got = mx.attn_select(q.to(dev()), cu, index, table.to(dev()), torch.tensor([P * page], dtype=torch.int32, device=dev()), n_sel)
    want = long_ref.select(q, [nodes], codes, exps, table, [P * page], page, n_sel, 1, 1, nodes)
    assert torch.equal(got.cpu(), want)

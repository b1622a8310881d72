"""A sequence's last page, full or not, can be named to attn_sparse; the one after it names none, and is reported."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import test_gpu_attn_sparse as sparse

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,nodes", [(64, 1), (65, 1), (128, 3), (1000, 9), (1, 2)])
def test_last_page_and_the_next(ctx, nodes):
    c = sparse.Case([ctx], [nodes], 8, 1, 64, 64, 2, seed=4)
    last = -(-ctx // 64) - 1
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    c.sel[..., 0], c.sel[..., 1] = last, -1
    want = c.run(dev_status=status)
    c.check(want, "the last page")
    assert mx.mxg_query_status(status) == 0
    c.sel[..., 1] = last + 1
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 5

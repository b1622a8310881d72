"""The bounded waits of the attention kernels: debug_stall makes the first wait
of every CTA one that nothing satisfies; the kernel gives up, reports
MXG_DEV_TIMEOUT and returns, and the next call is right."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from test_gpu_attn_prompt import check, inputs, offsets
from test_gpu_attn_tree import Case
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_stall(D):
    d = dev()
    lens = [300, 5, 1000]
    q, k, v = inputs(1, sum(lens), 8, 2, D, d)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    mx.attn_prompt(q, k, v, offsets(lens, d), dev_status=status, timeout_ms=20, debug_stall=1)
    assert mx.mxg_query_status(status) == 6
    out = mx.attn_prompt(q, k, v, offsets(lens, d), dev_status=status)
    assert mx.mxg_query_status(status) == 0
    check(out, q, k, v, lens, D ** -0.5, "after the timeout")


@pytest.mark.parametrize("nodes", [[4, 8, 1], [64, 40, 64]])
def test_tree_stall(nodes):
    c = Case([3000, 0, 500], nodes, 16, 2, 128, 64, seed=3)
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    c.run(dev_status=status, timeout_ms=20, debug_stall=1)
    assert mx.mxg_query_status(status) == 6
    out = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 0
    c.check(out, "after the timeout")

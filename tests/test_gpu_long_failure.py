"""The bounded waits of the long-context kernels: debug_stall makes the first wait of every CTA one that nothing
satisfies; the kernels give up, report MXG_DEV_TIMEOUT and return, and the next call is right."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import test_gpu_attn_shared as shared
import test_gpu_attn_sparse as sparse

pytestmark = pytest.mark.gpu

CASES = [
    (shared, ([2], [512], [300, 0, 500], [1, 1, 1], 16, 2, 128, 64)),
    (shared, ([2], [512], [300, 0, 500], [4, 8, 1], 16, 2, 64, 64)),
    (shared, ([3], [512], [300, 0, 500], [64, 40, 64], 16, 2, 128, 64)),
    (shared, ([48], [512], [7 * i % 300 for i in range(48)], [1] * 48, 8, 4, 64, 64)),  # (two launches beside one another)
    (shared, ([48], [512], [7 * i % 300 for i in range(48)], [3] * 48, 32, 4, 128, 64)),
    (sparse, ([3000, 0, 500], [1, 1, 1], 16, 2, 128, 64, 6)),
    (sparse, ([3000, 0, 500], [4, 8, 1], 16, 2, 64, 64, 6)),
    (sparse, ([3000, 0, 500], [64, 40, 64], 16, 2, 128, 64, 6)),
]


@pytest.mark.parametrize("module,args", CASES)
def test_stall(module, args):
    c = module.Case(*args, seed=3)
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    c.run(dev_status=status, timeout_ms=20, debug_stall=1)
    assert mx.mxg_query_status(status) == 6
    out = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 0
    c.check(out, "after the timeout")

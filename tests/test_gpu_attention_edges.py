"""The attention operators at the edges of what they take: tables without
columns."""
import math

import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev
from test_gpu_attn_tree import offsets, randn, tree_masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes", [[3], [5, 1, 64], [2, 0, 7] * 14])
def test_tree_a_table_without_columns(D, nodes):
    """Nothing is cached yet and the block table has no columns (its pointer is
    null): the nodes see one another, and nobody reads the table."""
    d = dev()
    N, B, Hq, Hkv = sum(nodes), len(nodes), 8, 2
    q, k, v = randn(1, N, Hq, D).to(d), randn(2, N, Hkv, D).to(d), randn(3, N, Hkv, D).to(d)
    mask = tree_masks(nodes, 4).to(d)
    kc = torch.zeros(1, 16, Hkv, D, dtype=torch.bfloat16, device=d)
    tab = torch.empty(B, 0, dtype=torch.int32, device=d)
    assert tab.data_ptr() == 0
    status = torch.zeros(1, dtype=torch.int32, device=d)
    out = mx.attn_tree(q, k, v, offsets(nodes, d), mask, mx.KVCache(kc, kc.clone()), tab,
                       torch.zeros(B, dtype=torch.int32, device=d), dev_status=status)
    assert mx.mxg_query_status(status) == 0
    for at, o, b in attn_ref.tree(q, k, v, nodes, mask, kc, kc, tab, [0] * B, 1 / math.sqrt(D)):
        attn_ref.assert_within(out[at], o, b, f"{nodes} D={D}")

"""The attention operators at the edges of what they take: tables without
columns, accepted nodes that cannot be written."""
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


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
def test_append_counts_only_what_it_writes(D, page):
    """An entry that cannot be written (no such node, no page in the table, a
    page outside the cache) ends its list: what follows is not written either,
    ctx_out holds the tokens that are in the cache, and the call reports it."""
    d = dev()
    layers, Hkv, pages, most = 2, 2, 12, 70
    nodes = [72, 4, 4, 4, 4, 3]
    tab = torch.tensor([[0, 1, 2, 3, 4], [5, -1, 6, 6, 6], [7, 99, 6, 6, 6], [8, 9, 10, 11, 6], [-3, 6, 6, 6, 6],
                        [6, 6, 6, 6, 6]], dtype=torch.int32)
    ctx = [1, page - 2, page - 1, 5 * page - 1, 0, 4]
    acc = torch.full((6, most), -1, dtype=torch.int32)
    acc[0] = torch.arange(most, dtype=torch.int32)
    acc[0, 66] = 72                                               # no such node, in the second round of 64 rows
    acc[1, :4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)    # the third token has no page
    acc[2, :3] = torch.tensor([0, 1, 3], dtype=torch.int32)       # the second token's page is not in the cache
    acc[3, :1] = 4                                                # no such node, and the table ends after this token
    acc[4, :2] = torch.tensor([0, 1], dtype=torch.int32)          # no page at all
    acc[5, :4] = torch.tensor([0, 7, 1, 2], dtype=torch.int32)    # no such node in the middle of the list
    take = [66, 2, 1, 0, 0, 1]
    cu = torch.tensor([0] + nodes).cumsum(0).int()
    N = int(cu[-1])
    kc, vc = (randn(s, layers, pages, page, Hkv, D).to(d) for s in (1, 2))
    k, v = (randn(s, layers, N, Hkv, D).to(d) for s in (3, 4))
    wk, wv = kc.clone(), vc.clone()
    for b, n in enumerate(take):
        for i in range(n):
            at = ctx[b] + i
            wk[:, int(tab[b, at // page]), at % page] = k[:, int(cu[b] + acc[b, i])]
            wv[:, int(tab[b, at // page]), at % page] = v[:, int(cu[b] + acc[b, i])]
    status = torch.zeros(1, dtype=torch.int32, device=d)
    got = mx.kv_append(k, v, cu.to(d), acc.to(d), mx.KVCache(kc, vc), tab.to(d),
                       torch.tensor(ctx, dtype=torch.int32, device=d), dev_status=status)
    assert mx.mxg_query_status(status) == 5
    assert got.tolist() == [c + n for c, n in zip(ctx, take)]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    # a list that ends by a negative entry right before a bad one reports nothing
    got = mx.kv_append(k, v, cu.to(d), torch.tensor([[0, -1, 500]] * 6, dtype=torch.int32, device=d), mx.KVCache(kc, vc),
                       torch.arange(6, dtype=torch.int32, device=d)[:, None], torch.zeros(6, dtype=torch.int32, device=d),
                       dev_status=status)
    assert mx.mxg_query_status(status) == 0 and got.tolist() == [1] * 6

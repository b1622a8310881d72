"""kv_index writes an entry a (layer, page, kv head): an index whose entries would lie over one another is refused, whichever
strides do it together; any order of layers, pages and heads is taken."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from test_attention_args import C
from test_attention_long_args import INDEX, X

two = dict(cache=C(layers=2))
OVER = [
    dict(index=X(codes_page=256, codes_head=256)),                             # page 1 head 0 is page 0 head 1
    dict(index=X(codes_page=496, codes_head=256)),                             # and half of it
    dict(index=X(codes_page=256, codes_head=768)),                             # heads around three of four pages
    dict(two, index=X(layers=2, codes_layer=2048, exps_layer=32)),             # layer 1 page 0 is layer 0 page 1
    dict(two, index=X(layers=2, codes_layer=6144, exps_layer=32)),             # and its page 3
    dict(two, index=X(layers=2, codes_layer=256, exps_layer=32)),              # and its head 1
    dict(two, index=X(layers=2, codes_layer=8192, exps_layer=8)),              # exponents: layer 1 page 0 is layer 0 page 1
    dict(two, index=X(layers=2, codes_layer=8192, exps_layer=3, exps_page=2)),
    dict(index=X(pages=(1 << 31) - 1, codes_page=(1 << 31) - 16, codes_head=1 << 37)),  # (2^62 bytes of pages)
]


@pytest.mark.parametrize("i", range(len(OVER)))
def test_entries_over_one_another_are_refused(i):
    assert mx.lib().kv_index(*{**INDEX, **OVER[i]}.values()) == 2


ORDERS = [(0, 1, 2), (1, 0, 2), (2, 1, 0), (0, 2, 1), (1, 2, 0), (2, 0, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("order", ORDERS)
def test_any_order_of_layers_pages_and_heads(order):
    L, P, H, D, page = 3, 5, 2, 64, 16
    g = torch.Generator().manual_seed(3)
    k = torch.randn(L, P, page, H, D, generator=g).bfloat16().cuda()
    cache = mx.KVCache(k, k)
    table = torch.tensor([[4, 0, 2], [1, 3, -1]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([48, 33], dtype=torch.int32, device="cuda")
    want = mx.kv_index(cache, mx.PageIndex.of(cache), table, None, ctx)
    back = [order.index(i) for i in range(3)]
    shape = [(L, P, H)[i] for i in order]
    codes = torch.zeros(*shape, 2, D, dtype=torch.int8, device="cuda").permute(*back, 3, 4)
    exps = torch.zeros(L, P, H, dtype=torch.uint8, device="cuda")
    if order.index(0) > order.index(1):
        exps = torch.zeros(P, L, H, dtype=torch.uint8, device="cuda").transpose(0, 1)
    got = mx.kv_index(cache, mx.PageIndex(codes, exps, page), table, None, ctx)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.exps, want.exps) and bool(want.exps.any())

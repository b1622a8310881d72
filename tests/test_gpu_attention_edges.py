"""The attention operators at the edges of what they take: tables without
columns, accepted nodes that cannot be written, rows that one key has nearly all of,
caches of several layers, limits of the waits that are none,
results in place of q."""
import math

import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev
from test_gpu_attn_tree import Case, offsets, randn, tree_masks

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


# One key has nearly all of a row, and comes after the running reference was
# set by another: its weight is 2^x, x between 5 and 8, not 1, and is rounded to
# bf16 for the product.  The values are alike over the keys, so the row's result
# is that value: exactly, if the heavy weight's rounding is in the sum too.
# What else there is: the first key's weight, 1, and a few hundred of at most
# 2^-20, whose roundings move the result by 2^-25; the fp32 sums by 300 2^-23;
# half a unit of bf16 is 2^-9.

def heavy_key(T, H, D, first, heavy, seed):
    """Keys (T, H, D) along one direction: 0 at `first`, 1 at `heavy`, else -4;
    and queries' lengths along it for scores of 3.6 to 5.4 with the heavy one."""
    k = torch.full((T, H, 1), -4.0)
    k[first], k[heavy] = 0.0, 1.0
    e = torch.zeros(D)
    e[seed % D] = 1.0
    return (k * e).bfloat16(), e


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [([600, 420], 8, 2), ([400] * 5, 8, 8), ([300] * 40, 2, 1)])
def test_prompt_one_heavy_key(D, lens, Hq, Hkv):
    d = dev()
    T, at = sum(lens), 0
    g = torch.Generator().manual_seed(T + D)
    q = (3.6 + 1.8 * torch.rand(T, Hq, 1, generator=g)).bfloat16()
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16)
    rows = []
    for n in lens:
        j = 128 + int(torch.randint(0, n - 130, (1,), generator=g))
        k[at:at + n], e = heavy_key(n, Hkv, D, 0, j, 3)
        rows += range(at + j, at + n)
        at += n
    one = randn(33, 1, Hkv, D).to(d)
    out = mx.attn_prompt((q * e).bfloat16().to(d), k.to(d), one.expand(T, -1, -1).contiguous(), offsets(lens, d), scale=1.0)
    off = out[rows] != one.repeat_interleave(Hq // Hkv, 1)
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} values are not the value"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n,ctx", [(40, 3, 300), (100, 16, 130)])
def test_tree_one_heavy_key(D, B, n, ctx):
    """Every node sees the context and itself; its own key is the heavy one."""
    Hq, Hkv, page = 16, 8, 32
    c = Case([ctx] * B, [n] * B, Hq, Hkv, D, page, seed=36)
    d = c.q.device
    kc, e = heavy_key(ctx, Hkv, D, 0, 0, 5)
    kc[0] = 0
    j = torch.arange(ctx)
    for b in range(B):
        c.kc[c.tab[b].long()[(j // page).to(d)], (j % page).to(d)] = kc.to(d)
    g = torch.Generator().manual_seed(D + B)
    N = B * n
    c.q = ((3.6 + 1.8 * torch.rand(N, Hq, 1, generator=g)).bfloat16() * e).bfloat16().to(d)
    c.k = e.bfloat16().expand(N, Hkv, D).contiguous().to(d)
    c.mask = torch.tensor([1 << i for i in range(n)] * B, dtype=torch.int64, device=d)
    one = randn(35, 1, Hkv, D).to(d)
    c.v = one.expand(N, -1, -1).contiguous()
    c.vc = one[0].expand(c.vc.shape).contiguous()
    off = c.run(scale=1.0) != one.repeat_interleave(Hq // Hkv, 1)
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} values are not the value"


def test_calls_of_one_layer_refuse_a_cache_of_several():
    """attn_tree and qk_norm_rope work on one layer: given a cache of three they
    do not silently take its first.  One layer of it, and a cache of one, are
    taken."""
    c = Case([40, 9], [3, 2], 4, 2, 64, 16, seed=37)
    d = c.q.device
    many = mx.KVCache(torch.stack([c.kc * 0, c.kc, c.kc * 0]), torch.stack([c.vc * 0, c.vc, c.vc * 0]))
    one = mx.KVCache(c.kc[None], c.vc[None])
    run = lambda cache: mx.attn_tree(c.q, c.k, c.v, c.cu, c.mask, cache, c.tab, c.len)  # noqa: E731
    want = c.run()
    assert torch.equal(run(many.layer(1)), want) and torch.equal(run(one), want)
    with pytest.raises(ValueError, match="layer"):
        run(many)
    keep = many.k.clone()
    slots = torch.arange(5, device=d)
    with pytest.raises(ValueError, match="layer"):
        mx.qk_norm_rope(c.q, c.k, v=c.v, cache=many, slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(many.k.nan_to_num(7.0), keep.nan_to_num(7.0))
    mx.qk_norm_rope(c.q, c.k, v=c.v, cache=many.layer(2), slots=slots)
    assert torch.equal(many.k[2, 0, :5], c.k) and torch.equal(many.k[:2].nan_to_num(7.0), keep[:2].nan_to_num(7.0))


@pytest.mark.parametrize("kw", [dict(timeout_ms=-1), dict(timeout_ms=1 << 32), dict(timeout_ms=(1 << 32) + 5),
                                dict(debug_stall=-1), dict(debug_stall=2), dict(debug_stall=1 << 32)])
def test_wait_limits_out_of_range_are_refused(kw):
    """-1 ms is not a limit of 49 days, nor 2^32 + 5 one of 5 ms."""
    c = Case([40, 9], [3, 2], 4, 2, 64, 16, seed=38)
    with pytest.raises(ValueError, match=next(iter(kw))):
        c.run(**kw)
    with pytest.raises(ValueError, match=next(iter(kw))):
        mx.attn_prompt(c.q, c.k, c.v, c.cu, **kw)
    mx.attn_prompt(c.q, c.k, c.v, c.cu, timeout_ms=(1 << 32) - 1)


@pytest.mark.parametrize("D", [64, 128])
def test_results_in_place_of_q(D):
    """out may be q itself: a row group's q is read by those that make its
    result, and written when all of them have it."""
    c = Case([9000, 300, 0, 2500], [8, 1, 40, 30], 16, 2, D, 64, seed=39)
    want, q = c.run(), c.q.clone()
    assert c.run(out=c.q) is c.q and torch.equal(c.q, want)
    lens = [1, 7, 1000, 300]
    qkv = randn(40, sum(lens), 20, D).to(q.device)
    q, k, v = qkv[:, :16], qkv[:, 16:18], qkv[:, 18:]
    cu = offsets(lens, q.device)
    want = mx.attn_prompt(q, k, v, cu)
    mx.attn_prompt(q, k, v, cu, out=q)
    assert torch.equal(q, want)

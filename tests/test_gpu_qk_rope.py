"""qk_norm_rope and kv_append against their definitions."""
import math

import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev

pytestmark = pytest.mark.gpu


def table(max_pos, rot, d):
    p = torch.arange(max_pos, dtype=torch.float64)
    a = p[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float().to(d).contiguous()


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", [
    (1, 64, 8, 128, 128, False, True), (64, 64, 8, 128, 128, False, True), (700, 64, 8, 128, 128, False, True),
    (7, 5, 1, 64, 64, False, True), (7, 5, 1, 64, 32, True, True), (33, 3, 3, 128, 64, True, True),
    (19, 2, 1, 16, 16, False, True), (19, 2, 1, 16, 16, True, True), (5, 7, 2, 24, 16, False, True),
    (5, 7, 2, 96, 96, False, True), (5, 7, 2, 192, 64, False, True), (5, 7, 2, 256, 256, False, True),
    (5, 7, 2, 256, 256, True, True), (5, 7, 2, 248, 240, False, True), (9, 4, 2, 128, 0, False, True),
    (9, 4, 2, 128, 128, False, False), (2000, 12, 2, 40, 32, False, True),
])
def test_norm_rope(T, Hq, Hkv, D, rot, inter, norm):
    d = dev()
    qkv = randn(T + D, T, Hq + 2 * Hkv, D, scale=3.0)
    qkv[:, :, ::7] *= 20
    qkv[T // 2, 0] = 0                      # a head of zeros
    qkv = qkv.to(d)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]  # slices of the packed projection
    wq, wk = (1 + randn(1, D, scale=0.3)).to(d), (1 + randn(2, D, scale=0.3)).to(d)
    if not norm:
        wq = wk = None
    cs = table(3000, rot, d) if rot else None
    pos = torch.randint(0, 3000, (T,), generator=torch.Generator().manual_seed(3)).int().to(d)
    pos[0] = 2999
    before = qkv.clone()
    qo, ko = mx.qk_norm_rope(q, k, pos, cs, wq=wq, wk=wk, eps=1e-5, interleaved=inter)
    assert torch.equal(qkv, before)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        attn_ref.assert_rounded(got, *attn_ref.norm_rope(x, w, 1e-5, cs, pos, inter), what)
    # in place, the same bits
    mx.qk_norm_rope(q, k, pos, cs, wq=wq, wk=wk, eps=1e-5, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_norm_of_one_tensor_only():
    d = dev()
    q, k = randn(4, 6, 4, 64).to(d), randn(5, 6, 2, 64).to(d)
    w = (1 + randn(6, 64, scale=0.3)).to(d)
    qo, ko = mx.qk_norm_rope(q, k, wq=w)
    attn_ref.assert_rounded(qo, *attn_ref.norm_rope(q, w, 1e-6, None, None, False), "q")
    assert torch.equal(ko, k)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,head_major", [(1, 8, 1, 128, 16, False), (300, 64, 8, 128, 64, False),
                                                        (77, 6, 3, 64, 32, True), (50, 2, 2, 96, 256, False)])
def test_rope_into_the_cache(T, Hq, Hkv, D, page, head_major):
    """k and v land in their slots and nowhere else; negative slots are not written."""
    d = dev()
    pages = T // page + 3
    shape = (pages, Hkv, page, D) if head_major else (pages, page, Hkv, D)
    kc, vc = randn(7, *shape).to(d), randn(8, *shape).to(d)
    if head_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    q, k, v = randn(9, T, Hq, D).to(d), randn(10, T, Hkv, D).to(d), randn(11, T, Hkv, D).to(d)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(12))[:T].to(d)
    slots[::5] = -1
    cs, pos = table(500, D // 16 * 16, d), torch.arange(T, device=d).int()
    w = (1 + randn(13, D, scale=0.3)).to(d)
    want_k, want_v = kc.clone(), vc.clone()
    status = torch.zeros(1, dtype=torch.int32, device=d)
    _, ko = mx.qk_norm_rope(q, k, pos, cs, wq=w, wk=w, v=v, cache=mx.KVCache(kc, vc), slots=slots, dev_status=status)
    live = slots >= 0
    want_k[slots[live] // page, slots[live] % page] = ko[live]
    want_v[slots[live] // page, slots[live] % page] = v[live]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert mx.mxg_query_status(status) == 0


def test_rope_out_of_range_positions_and_slots():
    """A position outside the table makes the token NaN, a slot past the cache
    is not written; both are reported, the other tokens are right."""
    d = dev()
    T, H, D = 6, 2, 64
    q, k, v = randn(1, T, H, D).to(d), randn(2, T, H, D).to(d), randn(3, T, H, D).to(d)
    cs, pos = table(10, 64, d), torch.tensor([0, 9, 10, -1, 3, 2 ** 31 - 1], dtype=torch.int32, device=d)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    qo, ko = mx.qk_norm_rope(q, k, pos, cs, dev_status=status)
    assert mx.mxg_query_status(status) == 5
    bad = torch.tensor([2, 3, 5], device=d)
    good = torch.tensor([0, 1, 4], device=d)
    assert bool(torch.isnan(qo[bad]).all()) and bool(torch.isnan(ko[bad]).all())
    attn_ref.assert_rounded(qo[good], *attn_ref.norm_rope(q[good], None, 0, cs, pos[good], False), "q")
    kc, vc = torch.zeros(2, 16, H, D, dtype=torch.bfloat16, device=d), torch.zeros(2, 16, H, D, dtype=torch.bfloat16, device=d)
    slots = torch.tensor([0, 31, 32, 2 ** 62, -5, 7], device=d)
    mx.qk_norm_rope(q, k, v=v, cache=mx.KVCache(kc, vc), slots=slots, dev_status=status)
    assert mx.mxg_query_status(status) == 5
    flat = vc.view(32, H, D)
    assert torch.equal(flat[[0, 31, 7]], v[[0, 1, 5]]) and int((flat != 0).any(-1).any(-1).sum()) == 3


def test_rope_special_values_stay_in_their_head():
    d = dev()
    q, k = randn(1, 3, 4, 128).to(d), randn(2, 3, 2, 128).to(d)
    w = torch.ones(128, dtype=torch.bfloat16, device=d)
    ref, _ = mx.qk_norm_rope(q, k, wq=w, wk=w)
    q[1, 2, 5] = float("nan")
    got, _ = mx.qk_norm_rope(q, k, wq=w, wk=w)
    assert bool(torch.isnan(got[1, 2]).all())
    got[1, 2] = ref[1, 2]
    assert torch.equal(got, ref)


def test_rope_no_tokens_and_another_stream():
    d = dev()
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=d)
    qo, ko = mx.qk_norm_rope(e, e, torch.empty(0, dtype=torch.int32, device=d), table(4, 64, d))
    assert qo.shape == (0, 4, 64)
    q, k = randn(1, 50, 4, 64).to(d), randn(2, 50, 4, 64).to(d)
    pos, cs = torch.arange(50, device=d).int(), table(64, 64, d)
    want = mx.qk_norm_rope(q, k, pos, cs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mx.qk_norm_rope(q, k, pos, cs, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("layers,page,Hkv,D,most", [(1, 16, 8, 128, 8), (3, 64, 1, 64, 1), (2, 32, 3, 24, 70),
                                                    (5, 256, 2, 128, 5)])
def test_append(layers, page, Hkv, D, most):
    d = dev()
    ctx = [0, 1, page - 1, page, 3 * page + 5, 17]
    nodes = [most, 3, 0, most + 2, most + 1, 64 + most]
    B, N = len(ctx), sum(nodes)
    cols = max(c + most for c in ctx) // page + 1
    pages = B * cols + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(5))
    tab = order[:B * cols].view(B, cols).int().to(d)
    kc, vc = randn(1, layers, pages, page, Hkv, D).to(d), randn(2, layers, pages, page, Hkv, D).to(d)
    k, v = randn(3, layers, N, Hkv, D).to(d), randn(4, layers, N, Hkv, D).to(d)
    g = torch.Generator().manual_seed(6)
    acc = torch.full((B, most), -1, dtype=torch.int32)
    for b, n in enumerate(nodes):
        path = torch.randperm(n, generator=g)[:most].sort().values if n else torch.empty(0, dtype=torch.long)
        path = path[:len(path) - b % 2]
        acc[b, :len(path)] = path.int()
    if most > 2:
        acc[0, 2:] = -1
        acc[0, 3:] = 10 ** 6                 # past the end of the list: nobody's
    cu = torch.tensor([0] + nodes).cumsum(0).int()
    wk, wv, want_ctx = kc.clone(), vc.clone(), []
    for b, c in enumerate(ctx):
        i = 0
        while i < most and acc[b, i] >= 0:
            at = c + i
            wk[:, int(tab[b, at // page]), at % page] = k[:, int(cu[b] + acc[b, i])]
            wv[:, int(tab[b, at // page]), at % page] = v[:, int(cu[b] + acc[b, i])]
            i += 1
        want_ctx.append(c + i)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    got = mx.kv_append(k, v, cu.to(d), acc.to(d), mx.KVCache(kc, vc), tab, torch.tensor(ctx, dtype=torch.int32, device=d),
                       dev_status=status)
    assert torch.equal(kc, wk) and torch.equal(vc, wv) and got.tolist() == want_ctx
    assert mx.mxg_query_status(status) == 0


def test_append_out_of_range():
    d = dev()
    kc, vc = torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device=d), torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device=d)
    k, v = randn(1, 5, 1, 64).to(d), randn(2, 5, 1, 64).to(d)
    tab = torch.tensor([[0, -1], [1, 9], [2, 3]], dtype=torch.int32, device=d)
    ctx = torch.tensor([15, 16, 31], dtype=torch.int32, device=d)   # second token without a page / bad page / past the table
    acc = torch.tensor([[0, 1], [0, -1], [0, 5]], dtype=torch.int32, device=d)
    cu = torch.tensor([0, 2, 4, 5], dtype=torch.int32, device=d)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    mx.kv_append(k, v, cu, acc, mx.KVCache(kc, vc), tab, ctx, dev_status=status)
    assert mx.mxg_query_status(status) == 5
    want = torch.zeros_like(kc)
    want[0, 15], want[3, 15] = k[0], k[4]
    assert torch.equal(kc, want)


def test_append_nothing():
    d = dev()
    kc, vc = randn(1, 2, 16, 1, 64).to(d), randn(2, 2, 16, 1, 64).to(d)
    keep = kc.clone()
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=d)
    ctx = torch.tensor([3], dtype=torch.int32, device=d)
    got = mx.kv_append(e, e, torch.zeros(2, dtype=torch.int32, device=d), torch.full((1, 4), -1, dtype=torch.int32, device=d),
                       mx.KVCache(kc, vc), torch.zeros(1, 1, dtype=torch.int32, device=d), ctx)
    assert got.tolist() == [3] and torch.equal(kc, keep)

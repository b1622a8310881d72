"""qk_norm_rope where a head does not fill its lanes (D is not 16 times a power
of two, or rot leaves an odd number of units), both pairings: what lies beside a
head is neither read nor written."""
import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev
from test_gpu_qk_rope import randn, table

pytestmark = pytest.mark.gpu

WIDTHS = [(24, 16), (40, 32), (40, 16), (48, 48), (96, 96), (104, 48), (136, 128), (192, 64), (248, 240), (232, 16)]


def padded(x, value):
    """x (T, H, D) as the middle of rows of D + 16, the rest `value`."""
    T, H, D = x.shape
    buf = torch.full((T, H, D + 16), value, dtype=x.dtype, device=x.device)
    buf[:, :, 8:8 + D] = x
    return buf, buf[:, :, 8:8 + D]


def untouched(buf, D, value):
    rest = torch.cat([buf[..., :8], buf[..., 8 + D:]], -1).float()
    return bool((rest.isnan() if value != value else rest == value).all())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", WIDTHS)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 3, 1), (37, 5, 2), (700, 7, 1)])
def test_widths_that_do_not_fill_their_lanes(T, Hq, Hkv, D, rot, inter):
    d = dev()
    nan = float("nan")
    x = randn(T + D + rot, T, Hq + Hkv, D, scale=3.0).to(d)
    wq, wk = (1 + randn(1, D, scale=0.3)).to(d), (1 + randn(2, D, scale=0.3)).to(d)
    cs = table(900, rot, d)
    pos = torch.randint(0, 900, (T,), generator=torch.Generator().manual_seed(3)).int().to(d)
    (qb, q), (kb, k) = padded(x[:, :Hq], nan), padded(x[:, Hq:], nan)
    (qob, qo), (kob, ko) = padded(torch.zeros_like(q), 7.0), padded(torch.zeros_like(k), 7.0)
    mx.qk_norm_rope(q, k, pos, cs, wq=wq, wk=wk, eps=1e-5, interleaved=inter, q_out=qo, k_out=ko)
    for got, a, w, what in ((qo, x[:, :Hq], wq, "q"), (ko, x[:, Hq:], wk, "k")):
        attn_ref.assert_rounded(got, *attn_ref.norm_rope(a, w, 1e-5, cs, pos, inter), what)
    assert untouched(qob, D, 7.0) and untouched(kob, D, 7.0)
    assert torch.equal(q, x[:, :Hq]) and torch.equal(k, x[:, Hq:])
    # in place, the same bits
    mx.qk_norm_rope(q, k, pos, cs, wq=wq, wk=wk, eps=1e-5, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and untouched(qb, D, nan) and untouched(kb, D, nan)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page", [(90, 4, 2, 64, 32, 16), (300, 8, 2, 128, 128, 64), (50, 3, 1, 96, 96, 32),
                                                 (33, 2, 2, 24, 16, 16), (33, 2, 1, 248, 240, 16)])
def test_neighbouring_pairs_into_the_cache(T, Hq, Hkv, D, rot, page):
    """The cache has k as k_out has it, v as it is, and nothing else changes."""
    d = dev()
    pages = T // page + 3
    (kb, kc), (vb, vc) = (padded(randn(s, pages * page, Hkv, D).to(d), 7.0) for s in (4, 5))
    kc, vc = (c.view(pages, page, Hkv, D) for c in (kc, vc))
    q, k, v = randn(6, T, Hq, D).to(d), randn(7, T, Hkv, D).to(d), randn(8, T, Hkv, D).to(d)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(9))[:T].to(d)
    slots[1::4] = -1
    cs, pos, w = table(400, rot, d), torch.arange(T, device=d).int(), (1 + randn(10, D, scale=0.3)).to(d)
    want_k, want_v = kc.clone(), vc.clone()
    _, ko = mx.qk_norm_rope(q, k, pos, cs, wq=w, wk=w, interleaved=True, v=v, cache=mx.KVCache(kc, vc), slots=slots)
    attn_ref.assert_rounded(ko, *attn_ref.norm_rope(k, w, 1e-6, cs, pos, True), "k")
    live = slots >= 0
    want_k[slots[live] // page, slots[live] % page] = ko[live]
    want_v[slots[live] // page, slots[live] % page] = v[live]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert untouched(kb, D, 7.0) and untouched(vb, D, 7.0)

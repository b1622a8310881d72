"""attn_sparse where a v that only some nodes see is not finite: the others' rows are summed again from what they see."""
import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
import test_gpu_attn_sparse as sparse

pytestmark = pytest.mark.gpu

PAGE = 64


def poisoned(B, nodes, Hq, Hkv, D, channel, value, seed):
    """Sequences of four pages; node i names page i % 4, 0 and 3, so that 1 and 2 are seen by some; in page 1 a value."""
    c = sparse.Case([4 * PAGE] * B, [nodes] * B, Hq, Hkv, D, PAGE, 3, seed=seed)
    i = torch.arange(B * nodes, device=c.q.device) % nodes % 4
    c.sel[:] = torch.stack([torch.zeros_like(i), i, torch.full_like(i, 3)], 1).int()[:, None]
    for b in range(B):
        c.vc[int(c.tab[b, 1]), 5 + b % 50, b % Hkv, channel] = value
    return c


# items of a CTA each (three key tiles, as many strips as SMs or twice that), and items that several share
BATCHES = {"whole": (lambda sms: max(sms // 8, 1), 8), "two": (lambda sms: max(sms // 4, 1), 8), "shared": (lambda sms: 2, 4)}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("channel,value", [(1, "nan"), (-2, "nan"), (-1, "inf")])
def test_in_place_of_q(D, batch, channel, value):
    many, Hkv = BATCHES[batch]
    B = many(torch.cuda.get_device_properties(0).multi_processor_count)
    c = poisoned(B, 10, 8 * Hkv, Hkv, D, channel, float(value), seed=80)
    want = c.run()
    seen = ~torch.isfinite(want[:, :, channel].float())
    assert bool(seen.any()) and bool(torch.isfinite(want[:, :, :-2][:, :, 2:].float()).all())
    c.q = c.q.clone()
    out = c.run(out=c.q)
    assert out.data_ptr() == c.q.data_ptr() and torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,nodes,Hq,Hkv", [(2, 10, 16, 2), (1, 64, 4, 1), (40, 9, 8, 1), (3, 3, 16, 2), (1, 20, 64, 1)])
def test_values_that_some_see(D, B, nodes, Hq, Hkv):
    for n, (channel, value) in enumerate([(3, float("nan")), (D - 1, float("-inf"))]):
        c = poisoned(B, nodes, Hq, Hkv, D, channel, value, seed=90 + n)
        c.v[nodes // 2, 0, 7] = float("nan")  # and a node's
        q = c.q.clone()
        c.check(c.run(), f"{B} {nodes} {Hq}/{Hkv} {channel} {value}")
        want = c.run()
        c.q = q.clone()
        assert torch.equal(c.run(out=c.q).view(torch.int16), want.view(torch.int16))
        c.q = q


@pytest.mark.parametrize("nodes", [8, 9])
def test_longest_lists(nodes):
    """512 pages of 256, two strips a CTA, one value of the newest page: no wait runs out.  (The table's rows name the
    same pages.)"""
    page, n_sel, G, D = 256, 512, 8, 128
    d = torch.device("cuda")
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device=d).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=d).bfloat16()  # noqa: E731
    kc, vc, N = rnd(n_sel + 1, page, 1, D), rnd(n_sel + 1, page, 1, D), B * nodes
    q, k, v = rnd(N, G, D), rnd(N, 1, D), rnd(N, 1, D)
    table = torch.arange(n_sel + 1, dtype=torch.int32, device=d).expand(B, -1).contiguous()
    ctx = torch.full((B,), (n_sel + 1) * page, dtype=torch.int32, device=d)
    cu = torch.arange(0, N + 1, nodes, dtype=torch.int32, device=d)
    sel = torch.arange(n_sel, dtype=torch.int32, device=d).expand(N, 1, -1).clone()
    sel[::nodes, 0, -1] = n_sel  # each first node's
    vc[n_sel, 3, 0, D - 1] = float("nan")
    mask, status = torch.ones(N, dtype=torch.int64, device=d), torch.zeros(1, dtype=torch.int32, device=d)
    out = mx.attn_sparse(q, k, v, cu, mask, mx.KVCache(kc, vc), table, ctx, sel, dev_status=status)
    assert mx.mxg_query_status(status) == 0
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[::nodes, :, D - 1] = True
    assert torch.equal(torch.isnan(out), nan)
    for a in (0, N - nodes):  # the first sequence's rows, the last one's
        for i in (a + 1, a + nodes - 1):
            ks = torch.cat([kc[:n_sel].reshape(-1, D), k[a]]).double()
            vs = torch.cat([vc[:n_sel].reshape(-1, D), v[a]]).double()
            o, bound = attn_ref.rows(q[i].double(), ks, vs, torch.ones(G, len(ks), dtype=torch.bool, device=d), D ** -0.5)
            attn_ref.assert_within(out[i], o, bound, f"node {i}")

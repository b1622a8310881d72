"""attn_sparse against softmax attention over the selected pages in 64 bits."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import long_ref
from gpu_util import dev
from test_gpu_attn_tree import Case as TreeCase, signed

pytestmark = pytest.mark.gpu


class Case(TreeCase):
    def __init__(self, ctx, nodes, Hq, Hkv, D, page, n_sel, seed=0, head_major=False, alike=0.5):
        super().__init__(ctx, nodes, Hq, Hkv, D, page, seed, head_major)
        g = torch.Generator().manual_seed(seed + 9)
        sel = torch.full((sum(nodes), Hkv, n_sel), -1, dtype=torch.int32)
        a = 0
        for c, n in zip(ctx, nodes):
            have = -(-c // page)
            common = torch.rand(Hkv, have, generator=g)
            for i in range(a, a + n):
                score = alike * common + (1 - alike) * torch.rand(Hkv, have, generator=g)
                m = min(n_sel, have)
                sel[i, :, :m] = score.topk(m, -1).indices.sort(-1).values.int()
            a += n
        self.sel = sel.to(dev())

    def run(self, **kw):
        return mx.attn_sparse(self.q, self.k, self.v, self.cu, self.mask, mx.KVCache(self.kc, self.vc), self.tab, self.len,
                              self.sel, **kw)

    def check(self, out, what):
        for at, o, b in long_ref.sparse(self.q, self.k, self.v, self.nodes, self.mask, self.kc, self.vc, self.tab, self.ctx,
                                        self.sel, self.scale):
            long_ref.assert_within(out[at], o, b, what)


SHAPES = [
    ([0], [1], 4, 1, 16, 4), ([1], [1], 8, 1, 16, 1), ([127], [1], 8, 8, 16, 3), ([128], [1], 64, 8, 64, 2),
    ([129, 0], [1, 1], 2, 1, 128, 2), ([1500], [8], 64, 8, 64, 5), ([1000, 17, 0, 640], [8, 8, 8, 8], 16, 2, 16, 12),
    ([260, 0, 33], [64, 64, 0], 8, 1, 32, 3), ([2511, 1512, 513], [5, 1, 33], 12, 4, 256, 2), ([900], [64], 32, 2, 64, 4),
    ([300, 5], [20, 64], 14, 2, 32, 6), ([700, 200], [3, 9], 71, 1, 16, 9), ([1290], [2], 128, 1, 64, 7),
    ([4000], [1], 10, 2, 16, 100), ([3000, 1, 700], [17, 2, 40], 24, 8, 128, 6), ([5000], [16], 8, 8, 32, 1),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,nodes,Hq,Hkv,page,n_sel", SHAPES)
def test_sparse(D, ctx, nodes, Hq, Hkv, page, n_sel):
    c = Case(ctx, nodes, Hq, Hkv, D, page, n_sel, seed=sum(ctx) + Hq)
    c.check(c.run(), f"{ctx} {nodes} {Hq}/{Hkv} D={D} page={page} sel={n_sel}")


def test_long_context():
    c = Case([60001, 100, 30000], [3, 2, 1], 4, 2, 128, 64, 40, seed=3)
    c.check(c.run(), "long")


def test_most_pages():
    c = Case([9000], [2], 4, 1, 64, 16, 512, seed=4, alike=0.0)
    c.check(c.run(), "512 pages")


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 600, (300,), generator=g).tolist()
    nodes = torch.randint(0, 4, (300,), generator=g).tolist()
    c = Case(ctx, nodes, 4, 2, 64, 32, 4, seed=2)
    c.check(c.run(), "many")


def test_lists_in_any_order():
    """Pages twice, negative ones between, past the end: each page once, or none."""
    c = Case([1000, 640], [6, 1], 8, 2, 128, 64, 5, seed=5)
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    want = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 0
    s = c.sel
    back = torch.cat([s.flip(-1), torch.full_like(s[..., :2], -3), s, s[..., :1]], -1).contiguous()
    c.sel = back
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 0
    c.sel = back.clone()
    c.sel[1, 1, 5], c.sel[6, 0, 6], c.sel[0, 0, 6] = 16, 1 << 30, 2147483647
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 5


def test_pages_outside_the_cache_are_zeros():
    c = Case([1000], [3], 8, 2, 128, 64, 5, seed=5)
    c.tab[0, int(c.sel[0, 0, 1])] = -4
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    c.check(c.run(dev_status=status), "outside")
    assert mx.mxg_query_status(status) == 5


def test_rows_that_see_nothing():
    c = Case([0, 700, 700], [4, 3, 1], 8, 2, 128, 64, 3, seed=6)
    c.mask = c.mask.clone()
    c.mask[0], c.mask[1], c.mask[5], c.mask[7] = 0, signed(1 << 63 | 1 << 5), 0, 0
    c.sel[5, 0], c.sel[7, 1] = -1, -1
    out = c.run()
    assert not out[0].any() and not out[1].any() and not out[5, :4].any() and not out[7, 4:].any()
    c.check(out, "empty rows")


def test_what_is_not_seen_has_no_influence():
    """NaN and infinities in pages and nodes that a row does not see."""
    c = Case([1500, 1500], [6, 1], 8, 2, 64, 32, 6, seed=9, alike=0.2)
    c.mask[:6] = torch.tensor([1, 2, 4, 8, 16, 32])
    c.v[2], c.v[4, 1, 3], c.k[5] = float("nan"), float("-inf"), float("nan")
    for i, (node, h) in enumerate([(0, 0), (1, 1), (3, 0)]):
        page = int(c.tab[0, int(c.sel[node, h, 2 + i])])
        c.vc[page, 3 + i, h, 5], c.vc[page, 20, h] = float("inf"), float("nan")
        c.kc[page, 7, h, 11] = float("nan")
    out = c.run()
    c.check(out, "poisoned pages")
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out).all())


def test_strides_scale_and_out():
    c = Case([300, 77], [6, 9], 6, 2, 64, 32, 4, seed=5, head_major=True)
    want = c.run()
    c.check(want, "head-major pages")
    qkv = torch.cat([c.q, c.k, c.v], 1)
    c.q, c.k, c.v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    out = torch.empty(6, 15, 64, dtype=torch.bfloat16, device=c.q.device).transpose(0, 1)
    assert torch.equal(c.run(out=out), want)
    ws = torch.empty(mx.mxg_attn_sparse_workspace_bytes(15, 2, 4, 64), dtype=torch.uint8, device=c.q.device).fill_(0xFF)
    assert torch.equal(c.run(ws=ws), want) and torch.equal(c.run(ws=ws), want)
    c.scale = 0.31
    c.check(c.run(scale=0.31), "scale")


def test_rows_past_the_last_sequence_stay():
    c = Case([300, 70], [2, 3], 8, 2, 128, 64, 3, seed=4)
    d = c.q.device
    pad = lambda t: torch.cat([t, torch.full((3, *t.shape[1:]), float("nan"), device=d, dtype=t.dtype)])  # noqa: E731
    c.q, c.k, c.v = pad(c.q), pad(c.k), pad(c.v)
    c.mask = torch.cat([c.mask, torch.full((3,), -1, device=d)])
    c.sel = torch.cat([c.sel, torch.full((3, 2, 3), 1 << 30, device=d, dtype=torch.int32)])
    out = torch.full((8, 8, 128), 7.0, dtype=torch.bfloat16, device=d)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    c.run(out=out, dev_status=status)
    assert bool((out[5:] == 7).all()) and mx.mxg_query_status(status) == 0
    c.check(out, "padded batch")


def test_all_pages_as_attn_tree():
    c = Case([1000, 333, 64], [5, 1, 9], 16, 2, 128, 64, 16, seed=8)
    c.check(c.run(), "all pages")
    TreeCase.check(c, c.run(), "all pages, as a tree")


def test_same_result_each_time_and_on_a_stream():
    c = Case([6000, 100, 3000], [8, 1, 64], 64, 8, 128, 64, 12, seed=14)
    want = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("nodes,scale", [([1, 1], 3.0), ([2, 1], 3.0), ([8, 5], 3.0), ([16, 3], 3.0), ([1, 1], 60.0), ([8, 3], 60.0)])
def test_scores_far_apart(nodes, scale):
    """Scores that differ by hundreds, the largest where they may: the reference has to be moved."""
    c = Case([900, 333], nodes, 8, 2, 128, 64, 9, seed=17)
    c.scale = scale
    for i, t in enumerate([0, 5, 64 * 3, 64 * 7 + 1, 899]):  # a key along a query each
        page = int(c.tab[0, t // 64])
        c.kc[page, t % 64, i % 2] = c.q[0, (i % 2) * 4 + i % 4] * (0.5 if i % 2 else 2.0)
    c.check(c.run(scale=scale), f"{nodes} {scale}")


@pytest.mark.parametrize("n", [1, 3, 8])
def test_first_key_that_counts_for_nothing(n):
    """A first key whose score is -infinity in 32 bits, or NaN, or infinite."""
    c = Case([300, 300], [n, n], 8, 2, 128, 64, 5, seed=19)
    for b in range(2):
        page = int(c.tab[b, 0])
        c.kc[page, 0, 0] = -c.q[b * n, 1].sign() * 3e38
    c.kc[int(c.tab[1, 0]), 0, 1] = float("nan")
    out = c.run()
    # the row that the key was made against has only negative products, a score of -infinity in 32 bits, and does without
    # it; the others' products of either sign overflow 32 bits, and what comes of infinity - infinity is theirs
    assert bool(torch.isfinite(out[0, 1].float()).all()) and bool(torch.isfinite(out[n, 1].float()).all())
    assert bool(torch.isnan(out[n:, 4:]).all())
    c.kc[:, 0, 0] = 0
    c.kc[int(c.tab[1, 0]), 0, 1] = 0
    c.check(c.run(), "after")


@pytest.mark.parametrize("nodes", [[1, 1], [4, 2], [8, 5], [40, 33]])
def test_large_values(nodes):
    """Values 2^76 times as large: the same bits with another exponent, whatever the reference of a row is."""
    c = Case([900, 333], nodes, 8, 2, 128, 64, 9, seed=23)
    for b in range(2):  # a first key far below the others of its rows
        c.kc[int(c.tab[b, 0]), 0] = -c.q[c.nodes[0] * b].view(2, 4, -1).float().mean(1).bfloat16()
    want = c.run()
    c.check(want, "as they are")
    c.v, c.vc = c.v * 2.0**76, c.vc * 2.0**76
    assert torch.equal(c.run(), want * 2.0**76)

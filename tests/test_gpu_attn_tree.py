"""attn_tree against softmax attention in 64 bits."""
import math

import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev

pytestmark = pytest.mark.gpu


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def offsets(lens, d):
    return torch.tensor([0] + list(lens)).cumsum(0).int().to(d)


def signed(w):
    return w - (1 << 64) if w >> 63 else w


def tree_masks(nodes, seed):
    """A random tree per sequence: every node sees its ancestors and itself."""
    g = torch.Generator().manual_seed(seed)
    words = []
    for n in nodes:
        row = []
        for i in range(n):
            up = row[int(torch.randint(0, i, (1,), generator=g))] if i else 0
            row.append(up | 1 << i)
        words += row
    return torch.tensor([signed(w) for w in words], dtype=torch.int64)


class Case:
    def __init__(self, ctx, nodes, Hq, Hkv, D, page, seed=0, head_major=False):
        d = dev()
        self.ctx, self.nodes, self.scale = ctx, nodes, 1 / math.sqrt(D)
        need = [-(-c // page) for c in ctx]
        cols, pages = max(max(need), 1) + 1, sum(need) + 3
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        tab = torch.full((len(ctx), cols), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            tab[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        shape = (pages, Hkv, page, D) if head_major else (pages, page, Hkv, D)
        self.kc, self.vc = randn(seed + 1, *shape).to(d), randn(seed + 2, *shape).to(d)
        if head_major:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        # what is in a page past the sequence's last token belongs to nobody
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, c in enumerate(ctx):
            for j in range(need[b]):
                used[tab[b, j], :min(page, c - j * page)] = True
        self.kc[~used.to(d)] = float("nan")
        self.vc[~used.to(d)] = float("nan")
        N = sum(nodes)
        self.q, self.k, self.v = randn(seed + 3, N, Hq, D, scale=1.5).to(d), randn(seed + 4, N, Hkv, D).to(d), \
            randn(seed + 5, N, Hkv, D).to(d)
        self.tab, self.mask, self.cu = tab.to(d), tree_masks(nodes, seed + 6).to(d), offsets(nodes, d)
        self.len = torch.tensor(ctx, dtype=torch.int32, device=d)

    def run(self, **kw):
        return mx.attn_tree(self.q, self.k, self.v, self.cu, self.mask, mx.KVCache(self.kc, self.vc), self.tab,
                            self.len, **kw)

    def check(self, out, what):
        for at, o, b in attn_ref.tree(self.q, self.k, self.v, self.nodes, self.mask, self.kc, self.vc, self.tab, self.ctx,
                                      self.scale):
            attn_ref.assert_within(out[at], o, b, what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,nodes,Hq,Hkv,page", [
    ([0], [1], 4, 1, 16), ([1], [1], 8, 1, 16), ([127], [1], 8, 8, 16), ([128], [1], 64, 8, 64), ([129, 0], [1, 1], 2, 1, 128),
    ([1500], [8], 64, 8, 64), ([1000, 17, 0, 640], [8, 8, 8, 8], 16, 2, 16), ([260, 0, 33], [64, 64, 0], 8, 1, 32),
    ([511, 512, 513], [5, 1, 33], 12, 4, 256), ([90], [64], 32, 2, 64), ([300, 5], [20, 64], 14, 2, 32),
    ([70, 200], [3, 9], 71, 1, 16), ([129], [2], 128, 1, 64), ([4000], [1], 10, 2, 16), ([3000, 1, 700], [17, 2, 40], 24, 8, 128),
])
def test_tree(D, ctx, nodes, Hq, Hkv, page):
    c = Case(ctx, nodes, Hq, Hkv, D, page, seed=sum(ctx) + Hq)
    c.check(c.run(), f"{ctx} {nodes} {Hq}/{Hkv} D={D} page={page}")


def test_tree_long_context():
    c = Case([40001, 100], [3, 2], 4, 2, 128, 64, seed=3)
    c.check(c.run(), "long")


def test_tree_many_sequences():
    g = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 300, (500,), generator=g).tolist()
    nodes = torch.randint(0, 4, (500,), generator=g).tolist()
    c = Case(ctx, nodes, 4, 2, 64, 32, seed=2)
    c.check(c.run(), "many")


def test_tree_pages_head_by_head_and_strided_nodes():
    c = Case([300, 77], [6, 9], 6, 2, 64, 32, seed=5, head_major=True)
    want = c.run()
    c.check(want, "head-major pages")
    qkv = torch.cat([c.q, c.k, c.v], 1)
    c.q, c.k, c.v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    out = torch.empty(6, 15, 64, dtype=torch.bfloat16, device=c.q.device).transpose(0, 1)
    assert torch.equal(c.run(out=out), want)


def test_tree_masks_that_leave_nothing():
    """Without cached tokens a node whose mask is empty gets 0; with them the
    context alone counts.  Bits past the tree are nobody's."""
    c = Case([0, 200, 0], [4, 4, 64], 8, 2, 128, 64, seed=6)
    m = c.mask.clone()
    m[0], m[1], m[5] = 0, signed(1 << 63 | 1 << 5), 0      # the second: only bits past the tree's four nodes
    m[8 + 10] = -1                                         # sees all 64
    m[8 + 63] = signed(1 << 63)
    c.mask = m
    out = c.run()
    assert bool((out[0] == 0).all()) and bool((out[1] == 0).all())
    c.check(out, "masks")


@pytest.mark.parametrize("D", [64, 128])
def test_tree_unseen_nan_has_no_part(D):
    """k and v of a node are NaN: only nodes that see it are."""
    c = Case([150, 20], [12, 8], 8, 2, D, 16, seed=7)
    ref = c.run()
    c.k[5], c.v[5] = float("nan"), float("nan")
    out = c.run()
    sees = ((c.mask >> 5) & 1).bool()
    sees[12:] = False
    assert bool(sees.any()) and torch.equal(out[~sees], ref[~sees])
    assert bool(torch.isnan(out[sees]).all())
    c.k[5] = 0
    c.v[5] = 0
    c.v[5, :, 7] = float("inf")
    out = c.run()
    assert torch.equal(out[~sees], ref[~sees])
    assert not bool(torch.isfinite(out[sees][:, :, 7]).any()) and bool(torch.isfinite(out[sees][:, :, 8:]).all())


def test_tree_offsets_past_32_bits():
    """A cache of more than 2^31 elements: its last pages are read right."""
    d = dev()
    page, Hkv, D = 64, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    kc = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=d)
    vc = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=d)
    c = Case([500], [3], 16, Hkv, D, page, seed=8)
    for j in range(8):
        src = int(c.tab[0, j])
        kc[pages - 1 - j], vc[pages - 1 - j] = c.kc[src], c.vc[src]
        c.tab[0, j] = pages - 1 - j
    c.kc, c.vc = kc, vc
    c.check(c.run(), "far pages")
    # and written there
    got = mx.kv_append(c.k, c.v, c.cu, torch.tensor([[0, 2]], dtype=torch.int32, device=d), mx.KVCache(kc, vc), c.tab, c.len)
    assert got.tolist() == [502]
    assert torch.equal(kc[pages - 8, 52:54], c.k[[0, 2]]) and torch.equal(vc[pages - 8, 52:54], c.v[[0, 2]])


def test_tree_out_of_range_entries():
    """A page outside the cache reads as zeros, a context past the table is
    clamped, nodes past the 64th are not written; all are reported."""
    c = Case([200, 40], [4, 3], 8, 2, 64, 32, seed=9)
    c.vc[c.vc != c.vc] = 0
    c.kc[c.kc != c.kc] = 0
    d = c.q.device
    status = torch.zeros(1, dtype=torch.int32, device=d)
    c.tab[0, 2] = 10 ** 6
    c.tab[1, 0] = -7
    out = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.check(out, "pages")
    c = Case([96], [2], 4, 2, 64, 32, seed=10)
    c.tab = c.tab[:, :3].contiguous()
    c.len += 1000
    out = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.check(out, "clamped context")
    c.len[:] = -4
    c.ctx = [0]
    out = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.check(out, "negative context")
    c = Case([30], [64], 4, 2, 64, 32, seed=11)
    q, k, v = (torch.cat([x, x[:6]]) for x in (c.q, c.k, c.v))
    out = torch.full_like(q, 7.0)
    mx.attn_tree(q, k, v, offsets([70], d), torch.cat([c.mask, c.mask[:6]]), mx.KVCache(c.kc, c.vc), c.tab, c.len, out=out,
                 dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.check(out[:64], "64 of 70 nodes")
    assert bool((out[64:] == 7.0).all())


def test_tree_repeats_streams_and_workspaces():
    """The parts of long contexts are joined in a fixed order: the same bits
    every time, whatever the workspace held."""
    c = Case([9000, 300, 2500], [8, 1, 30], 16, 2, 128, 64, seed=12)
    want = c.run()
    c.check(want, "split")
    ws = torch.full((mx.mxg_attn_tree_workspace_bytes(128),), 255, dtype=torch.uint8, device=want.device)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [c.run(ws=ws, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    e = torch.empty(0, 16, 128, dtype=torch.bfloat16, device=want.device)
    ek = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=want.device)
    got = mx.attn_tree(e, ek, ek, torch.zeros(4, dtype=torch.int32, device=want.device),
                       torch.empty(0, dtype=torch.int64, device=want.device), mx.KVCache(c.kc, c.vc), c.tab, c.len)
    assert got.shape == e.shape


def test_one_node_trees_are_decoding():
    """A tree of one node is the last row of the prompt that the cache holds."""
    d = dev()
    n, Hq, Hkv, D, page = 333, 16, 2, 128, 32
    q, k, v = randn(1, n, Hq, D).to(d), randn(2, n, Hkv, D).to(d), randn(3, n, Hkv, D).to(d)
    prompt = mx.attn_prompt(q, k, v, offsets([n], d))
    pages = n // page + 1
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=d) for _ in range(2))
    cache = mx.KVCache(kc, vc)
    mx.qk_norm_rope(q, k, v=v, cache=cache, slots=torch.arange(n, device=d))
    tab = torch.arange(pages, dtype=torch.int32, device=d)[None]
    out = mx.attn_tree(q[-1:], k[-1:], v[-1:], offsets([1], d), torch.ones(1, dtype=torch.int64, device=d), cache, tab,
                       torch.tensor([n - 1], dtype=torch.int32, device=d))
    # both are within their bound of the same row
    for at, o, b in attn_ref.prompt(q, k, v, [n], 1 / math.sqrt(D), lambda m: torch.tensor([m - 1])):
        attn_ref.assert_within(out, o, b, "decode")
        attn_ref.assert_within(prompt[at], o, b, "prompt")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_a_value_that_is_not_finite_leaves_its_row_s_others(D, bad):
    """One channel of a node's v is NaN or infinite: the nodes that see it have
    all other channels as if that one were finite."""
    c = Case([150, 20, 0], [12, 8, 64], 8, 2, D, 16, seed=9)
    ref = c.run()
    for at, heads, ch in ((5, 0, 7), (13, 1, D - 1), (30, 0, 0)):
        c.v[at, heads, ch] = bad
    out = c.run()
    hit = torch.zeros(out.shape, dtype=torch.bool, device=out.device)
    first = [0, 12, 20]
    for at, heads, ch in ((5, 0, 7), (13, 1, D - 1), (30, 0, 0)):
        b = max(i for i in range(3) if first[i] <= at)
        lo, hi = first[b], first[b] + c.nodes[b]
        hit[lo:hi, heads * 4:heads * 4 + 4, ch] = ((c.mask[lo:hi] >> (at - lo)) & 1).bool()[:, None]
    assert bool(hit.any()) and torch.equal(out[~hit], ref[~hit])
    assert not bool(torch.isfinite(out[hit]).any())


def test_tree_streams_side_by_side():
    """Calls on two streams at once, outputs and scratch from the allocator:
    neither disturbs the other, nor what the current stream allocates next."""
    a = Case([9000, 300, 2500], [8, 1, 30], 16, 2, 128, 64, seed=12)
    b = Case([4000, 5000], [3, 17], 16, 2, 128, 64, seed=13)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(6):
        for i, c in enumerate((a, b)):
            outs[i].append(c.run(stream=streams[i]))
        torch.full((24 << 20,), 1.0, device=a.q.device)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for got, w in zip(outs, want) for o in got)

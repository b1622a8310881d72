"""attn_shared against softmax attention in 64 bits."""
import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
import long_ref
from gpu_util import dev
from test_gpu_attn_tree import Case as TreeCase, signed

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


class Case(TreeCase):
    """tails: own cached tokens of each sequence; groups: sequences of each group, prefix: its shared tokens."""

    def __init__(self, groups, prefix, tails, nodes, Hq, Hkv, D, page, seed=0, head_major=False):
        own = [p for n, p in zip(groups, prefix) for _ in range(n)] + [0] * (len(tails) - sum(groups))
        super().__init__([t + p for t, p in zip(tails, own)], nodes, Hq, Hkv, D, page, seed, head_major)
        self.groups, self.prefix, self.page = groups, prefix, page
        # a group's other rows name nothing in their prefix: it is the first one's that is read
        b = 0
        for n, p in zip(groups, prefix):
            if n > 1:
                self.tab[b + 1:b + n, :p // page] = -5
            b += n
        self.cg, self.pl = ints([0] + torch.tensor(groups).cumsum(0).tolist() if groups else [0]), ints(prefix)

    def run(self, **kw):
        return mx.attn_shared(self.q, self.k, self.v, self.cu, self.mask, mx.KVCache(self.kc, self.vc), self.tab, self.len,
                              self.cg, self.pl, **kw)

    def check(self, out, what):
        tab = long_ref.shared_table(self.tab, self.groups, self.prefix, self.page)
        for at, o, b in attn_ref.tree(self.q, self.k, self.v, self.nodes, self.mask, self.kc, self.vc, tab, self.ctx,
                                      self.scale):
            attn_ref.assert_within(out[at], o, b, what)


SHAPES = [
    ([1], [64], [0], [1], 4, 1, 16),
    ([2], [128], [0, 0], [1, 1], 8, 8, 16),
    ([2], [128], [1, 0], [1, 1], 64, 8, 64),
    ([3], [144], [5, 17, 130], [2, 1, 3], 8, 1, 16),
    ([2, 3], [512, 0], [100, 300, 7, 0, 129], [8, 8, 8, 8, 8], 16, 2, 64),
    ([], [], [300, 0, 40], [3, 1, 2], 8, 2, 32),
    ([4], [1024], [64, 100, 185, 511], [8, 8, 8, 8], 64, 8, 64),
    ([3, 1, 2], [640, 128, 1280], [0, 5, 300, 17, 900, 2, 777, 0], [1, 20, 64, 3, 1, 31, 5, 0], 12, 4, 128),
    ([2, 2], [256, 256], [3, 0, 256, 1], [64, 64, 64, 1], 32, 2, 256),
    ([40], [160], [3 * i % 50 for i in range(40)], [1] * 40, 14, 2, 32),
    ([5], [3200], [11] * 5, [33, 1, 2, 64, 7], 71, 1, 64),
    ([3], [128], [10, 20, 30], [2, 0, 1], 128, 1, 64),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups,prefix,tails,nodes,Hq,Hkv,page", SHAPES)
def test_shared(D, groups, prefix, tails, nodes, Hq, Hkv, page):
    c = Case(groups, prefix, tails, nodes, Hq, Hkv, D, page, seed=sum(tails) + Hq)
    c.check(c.run(), f"{groups} {prefix} {tails} {nodes} {Hq}/{Hkv} D={D} page={page}")


def test_many_groups():
    g = torch.Generator().manual_seed(5)
    groups = torch.randint(0, 5, (150,), generator=g).tolist()
    B = sum(groups) + 20
    prefix = (torch.randint(0, 12, (150,), generator=g) * 32).tolist()
    tails = torch.randint(0, 150, (B,), generator=g).tolist()
    nodes = torch.randint(0, 4, (B,), generator=g).tolist()
    c = Case(groups, prefix, tails, nodes, 4, 2, 64, 32, seed=2)
    c.check(c.run(), "many")


def test_one_long_prefix():
    c = Case([30], [20480], [7 * i for i in range(30)], [1 + i % 3 for i in range(30)], 8, 2, 128, 64, seed=3)
    c.check(c.run(), "long")


def test_as_attn_tree_where_the_pages_are_the_same():
    c = Case([3, 2], [256, 640], [10, 0, 300, 64, 5], [4, 1, 9, 2, 2], 16, 2, 128, 64, seed=8)
    c.tab = long_ref.shared_table(c.tab, c.groups, c.prefix, c.page)
    out = c.run()
    c.check(out, "shared")
    TreeCase.check(c, TreeCase.run(c), "tree")
    # a prefix of no tokens
    c.pl, c.prefix = ints([0, 0]), [0, 0]
    c.check(c.run(), "nothing shared")


def test_strides_scale_and_out():
    c = Case([3], [128], [40, 77, 0], [6, 9, 2], 6, 2, 64, 32, seed=5, head_major=True)
    want = c.run()
    c.check(want, "head-major pages")
    qkv = torch.cat([c.q, c.k, c.v], 1)
    c.q, c.k, c.v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    out = torch.empty(6, 17, 64, dtype=torch.bfloat16, device=c.q.device).transpose(0, 1)
    assert torch.equal(c.run(out=out), want)
    ws = torch.empty(mx.mxg_attn_shared_workspace_bytes(17, 6, 64), dtype=torch.uint8, device=c.q.device).fill_(0xFF)
    assert torch.equal(c.run(ws=ws), want) and torch.equal(c.run(ws=ws), want)
    c.scale = 0.31
    c.check(c.run(scale=0.31), "scale")


def test_masks_that_leave_nothing():
    """A node without cached tokens whose mask is empty gets 0, in a group of no prefix and in none."""
    c = Case([2], [0], [0, 200, 0], [4, 4, 64], 8, 2, 128, 64, seed=6)
    m = c.mask.clone()
    m[0], m[1], m[5] = 0, signed(1 << 63 | 1 << 5), 0
    m[8 + 10], m[8 + 63], m[8 + 11] = -1, signed(1 << 63), 0
    c.mask = m
    out = c.run()
    assert not out[0].any() and not out[1].any() and not out[8 + 11].any()
    c.check(out, "empty masks")


def test_what_is_not_seen_has_no_influence():
    c = Case([2, 1], [128, 64], [30, 0, 200], [3, 5, 2], 8, 2, 64, 64, seed=9)
    c.mask[3:8] = torch.tensor([1, 2, 4, 8, 16])
    c.v[4], c.v[6, 1, 3], c.k[7] = float("nan"), float("inf"), float("nan")
    out = c.run()
    tab = long_ref.shared_table(c.tab, c.groups, c.prefix, c.page)
    every = torch.arange(tab.shape[1], dtype=torch.int32, device=tab.device).expand(10, 2, -1)
    for at, o, b in long_ref.sparse(c.q, c.k, c.v, c.nodes, c.mask, c.kc, c.vc, tab, c.ctx, every, c.scale):
        long_ref.assert_within(out[at], o, b, "poisoned nodes")


def test_rows_past_the_last_sequence_stay():
    c = Case([2], [64], [3, 70], [2, 3], 8, 2, 128, 64, seed=4)
    d = c.q.device
    pad = lambda t: torch.cat([t, torch.full((3, *t.shape[1:]), float("nan"), device=d, dtype=t.dtype)])  # noqa: E731
    c.q, c.k, c.v = pad(c.q), pad(c.k), pad(c.v)
    c.mask = torch.cat([c.mask, torch.full((3,), -1, device=d)])
    out = torch.full((8, 8, 128), 7.0, dtype=torch.bfloat16, device=d)
    c.run(out=out)
    assert bool((out[5:] == 7).all())
    c.check(out, "padded batch")


def test_offsets_out_of_range():
    """Groups and prefixes out of range are lowered, and reported; so are a page and a length."""
    c = Case([2, 2], [256, 128], [64, 0, 30, 10], [2, 3, 1, 4], 8, 2, 128, 64, seed=12)
    status = torch.zeros(1, dtype=torch.int32, device=c.q.device)
    want = c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 0
    c.pl = ints([400, 128])  # more than the second sequence's 256 tokens: its length
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 5
    c.pl = ints([256 + 63, 128])  # not whole pages
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 5
    c.pl, c.cg = ints([256, 128]), ints([0, 2, 9])  # past the last sequence
    assert torch.equal(c.run(dev_status=status), want) and mx.mxg_query_status(status) == 5
    c.cg, c.pl = ints([0, 2, 1]), ints([256, 999])  # falls: an empty group, and its length is nobody's
    c.run(dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.cg, c.pl, c.prefix = ints([-3, 2, 4]), ints([-1, 128]), [0, 128]
    c.tab[1, :4] = c.tab[0, :4]
    c.check(c.run(dev_status=status), "negative")
    assert mx.mxg_query_status(status) == 5
    c.cg, c.pl, c.prefix = ints([0, 2, 4]), ints([256, 128]), [256, 128]
    c.tab[0, 1] = 1 << 20  # a page of the prefix: zeros for the group
    c.check(c.run(dev_status=status), "a page outside")
    assert mx.mxg_query_status(status) == 5


def test_same_result_each_time_and_on_a_stream():
    c = Case([6], [2048], [5, 100, 700, 64, 0, 1], [8, 1, 3, 64, 2, 5], 64, 8, 128, 64, seed=14)
    want = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("nodes,scale", [([1, 1], 3.0), ([8, 5], 3.0), ([20, 64], 3.0), ([1, 1], 60.0), ([8, 3], 60.0)])
def test_scores_far_apart(nodes, scale):
    """Scores that differ by hundreds, in the prefix, in the own tokens and in the nodes."""
    c = Case([2], [512], [300, 40], nodes, 8, 2, 128, 64, seed=21)
    c.scale = scale
    for i, t in enumerate([0, 200, 511, 512, 700, 811]):
        page = int(c.tab[0, t // 64])
        c.kc[page, t % 64, i % 2] = c.q[0, (i % 2) * 4 + i % 4] * (0.5 if i % 2 else 2.0)
    c.k[nodes[0] - 1, 0] = c.q[nodes[0] - 1, 3] * 3
    c.check(c.run(scale=scale), f"{nodes} {scale}")


@pytest.mark.parametrize("nodes", [[1, 1], [4, 2], [8, 5], [40, 33]])
def test_large_values(nodes):
    """Values 2^76 times as large: the same bits with another exponent, whatever the reference of a row is."""
    c = Case([2], [512], [300, 40], nodes, 8, 2, 128, 64, seed=24)
    for b, t in ((0, 0), (0, 512), (1, 512)):  # first keys far below the others of their rows
        c.kc[int(c.tab[b, t // 64]), 0] = -c.q[c.nodes[0] * b].view(2, 4, -1).float().mean(1).bfloat16()
    want = c.run()
    c.check(want, "as they are")
    c.v, c.vc = c.v * 2.0**76, c.vc * 2.0**76
    assert torch.equal(c.run(), want * 2.0**76)


# more sequences x kv heads than SMs, few rows each: prefixes and sequences are launches of their own, beside one another
# where both are short (all but the last)
MANY = [
    ([48], [512], [7 * i % 300 for i in range(48)], [1] * 48, 8, 4, 64),
    ([20, 25], [1024, 160], [11 * i % 200 for i in range(50)], [i % 4 for i in range(50)], 16, 4, 32),
    ([], [], [i * 5 % 400 for i in range(160)], [1 + i % 3 for i in range(160)], 8, 1, 16),
    ([1, 30, 0, 2], [48, 2000, 16, 0], [3 * i % 170 for i in range(40)], [1 + (i == 7) * 63 for i in range(40)], 40, 8, 16),
    ([48], [12288], [37 * i % 509 for i in range(48)], [1] * 48, 64, 8, 64),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_many_sequences_of_few_rows(D, i):
    groups, prefix, tails, nodes, Hq, Hkv, page = MANY[i]
    c = Case(groups, prefix, tails, nodes, Hq, Hkv, D, page, seed=30 + i)
    out = c.run()
    c.check(out, MANY[i][:2])
    assert torch.equal(c.run(), out)


def test_many_sequences_scores_masks_and_values():
    """The same launches: scores far apart, masks that leave nothing, NaN that nobody sees, large values."""
    c = Case([30, 20], [256, 0], [13 * i % 300 for i in range(52)], [1 + i % 2 for i in range(52)], 8, 4, 128, 64, seed=40)
    c.scale = 3.0
    for i, t in enumerate([0, 100, 255, 256]):
        c.kc[int(c.tab[0, t // 64]), t % 64, i % 4] = c.q[0, (i % 4) * 2] * (0.5 if i % 2 else 2.0)
    c.mask[::3] = 0
    c.check(c.run(scale=3.0), "far apart")
    used = torch.zeros(c.kc.shape[0], dtype=torch.bool, device=dev())
    tab = long_ref.shared_table(c.tab, c.groups, c.prefix, c.page)
    for b, n in enumerate(c.ctx):
        used[tab[b, :-(-n // c.page)].long()] = True
    want = c.run(scale=3.0)
    c.kc[~used], c.vc[~used] = float("nan"), float("inf")
    for b, n in enumerate(c.ctx):
        if n % c.page:
            c.kc[int(tab[b, n // c.page]), n % c.page:] = float("nan")
            c.vc[int(tab[b, n // c.page]), n % c.page:] = float("nan")
    assert torch.equal(c.run(scale=3.0), want)
    c.vc[used] = torch.nan_to_num(c.vc[used], nan=0.0) * 2.0**76
    c.v = c.v * 2.0**76
    assert torch.equal(c.run(scale=3.0), want * 2.0**76)

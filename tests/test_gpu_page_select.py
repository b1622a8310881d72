"""kv_index and attn_select: bounds and choices are whole numbers, compared for equality."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import long_ref
from gpu_util import dev

pytestmark = pytest.mark.gpu


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def a_table(ctx, page, seed, more=3):
    need = [-(-c // page) for c in ctx]
    pages = sum(need) + more
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    tab = torch.full((len(ctx), max(max(need), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        tab[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return tab, pages


def an_index(seed, layers, pages, Hkv, D, page):
    """An index of arbitrary bytes: what is not written has to stay."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-128, 128, (layers, pages, Hkv, 2, D), generator=g, dtype=torch.int8).to(dev())
    exps = torch.randint(0, 256, (layers, pages, Hkv), generator=g, dtype=torch.uint8).to(dev())
    return mx.PageIndex(codes, exps, page)


def check_index(index, before, k, tab, old, new, page, what):
    codes, exps = before
    for b, (o, n) in enumerate(zip(old, new)):
        for j in range(o // page, n // page):
            pg = int(tab[b, j])
            if not 0 <= pg < k.shape[1]:
                continue
            for layer in range(k.shape[0]):
                for h in range(k.shape[3]):
                    codes[layer, pg, h], exps[layer, pg, h] = long_ref.bounds(k[layer, pg, :, h])
    assert torch.equal(index.exps.cpu(), exps), f"{what}: exps"
    assert torch.equal(index.codes.cpu(), codes), f"{what}: codes"


def copy_of(index):
    return index.codes.cpu().clone(), index.exps.cpu().clone()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layers,Hkv,page,old,new", [
    (1, 1, 16, [0], [0]), (1, 1, 16, [0], [15]), (1, 2, 16, [15], [16]), (2, 8, 64, [0, 63, 64], [64, 64, 64]),
    (3, 2, 32, [5, 0, 100, 7], [200, 31, 90, 8]), (1, 4, 128, [0, 127], [513, 129]), (2, 1, 256, [0], [1000]),
    (1, 3, 16, [3] * 40, [3 + 5 * i for i in range(40)]),
])
def test_index(D, layers, Hkv, page, old, new):
    tab, pages = a_table([max(o, n) for o, n in zip(old, new)], page, seed=sum(new))
    k = randn(sum(new) + D, layers, pages, page, Hkv, D)
    k[..., 5] *= 30
    k = k.to(dev())
    index = an_index(1, layers, pages, Hkv, D, page)
    before = copy_of(index)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    assert mx.kv_index(mx.KVCache(k, k), index, tab.to(dev()), ints(old), ints(new), dev_status=status) is index
    assert mx.mxg_query_status(status) == 0
    check_index(index, before, k.cpu(), tab, old, new, page, f"{old} {new} page={page}")


def test_index_of_many_sequences():
    g = torch.Generator().manual_seed(4)
    new = torch.randint(0, 90, (700,), generator=g).tolist()
    tab, pages = a_table(new, 16, 5)
    k = randn(6, 1, pages, 16, 2, 64).to(dev())
    index = an_index(2, 1, pages, 2, 64, 16)
    before = copy_of(index)
    mx.kv_index(mx.KVCache(k, k), index, tab.to(dev()), None, ints(new))
    check_index(index, before, k.cpu(), tab, [0] * 700, new, 16, "many")


def test_index_of_every_magnitude():
    """Zeros of both signs, the least and the largest numbers, exact powers of two, 127 and 127.5 of them, NaN, infinities."""
    top = [0.0, -0.0, 9.2e-41, -9.2e-41, 1e-38, 2.0 ** -101, 127 * 2.0 ** -100, 127.5 * 2.0 ** -100, 127.0, -127.0, 127.5,
           -127.5, 128.0, -128.0, 1.0, -1.0, 3.3895e38, -3.3895e38, 1.5e36, float("nan"), float("inf"), float("-inf")]
    page, D = 16, 64
    k = torch.zeros(1, len(top), page, 1, D)
    k[0, :, :, 0] = randn(3, page, D).float() * torch.tensor([abs(t) if abs(t) < 1e37 else 0.0 for t in top])[:, None, None] * 0.2
    for i, t in enumerate(top):
        k[0, i, i % page, 0, i] = t
        k[0, i, (i + 3) % page, 0, 50] = 1e-40  # counts as one step up
        k[0, i, :, 0, 51] = -1e-40
    k = k.nan_to_num(nan=float("nan"), posinf=float("inf"), neginf=float("-inf")).bfloat16().to(dev())
    index = an_index(3, 1, len(top), 1, D, page)
    before = copy_of(index)
    tab = torch.arange(len(top), dtype=torch.int32)[None]
    mx.kv_index(mx.KVCache(k, k), index, tab.to(dev()), ints([0]), ints([page * len(top)]))
    check_index(index, before, k.cpu(), tab, [0], [page * len(top)], page, "magnitudes")


def test_index_strides_and_ranges():
    """Pages head by head, an index inside a larger tensor, shared pages, numbers out of range."""
    page, D, Hkv, pages = 32, 128, 2, 9
    store = randn(8, 2, pages, Hkv, page, D).to(dev())
    k = store.transpose(2, 3)
    big = torch.zeros(2, pages + 2, Hkv, 3, 2 * D, dtype=torch.int8, device=dev())
    codes = big[:, :, :, 1].unflatten(-1, (2, D))
    exps = torch.full((2, pages + 2, 5), 9, dtype=torch.uint8, device=dev())
    index = mx.PageIndex(codes, exps[..., :Hkv], page)
    before = copy_of(index)
    tab = torch.tensor([[0, 1, 2, 3], [0, 1, 5, 6], [-1, 9, 8, 7]], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    mx.kv_index(mx.KVCache(k, k), index, tab.to(dev()), ints([0, 0, 0]), ints([127, 128, 128]), dev_status=status)
    assert mx.mxg_query_status(status) == 5  # (the pages -1 and 9)
    check_index(index, before, k.cpu(), tab, [0, 0, 0], [127, 128, 128], page, "strides")
    assert bool((exps[..., Hkv:] == 9).all()) and not big[:, :, :, 0].any() and not big[:, :, :, 2].any()
    before = copy_of(index)
    mx.kv_index(mx.KVCache(k, k), index, tab.to(dev()), ints([-5, 90, 1000]), ints([-1, 2000000000, 7]), dev_status=status)
    assert mx.mxg_query_status(status) == 5
    check_index(index, before, k.cpu(), tab, [0, 90, 128], [0, 128, 7], page, "ranges")


class Select:
    def __init__(self, ctx, nodes, Hq, Hkv, D, page, seed=0):
        d = dev()
        self.ctx, self.nodes, self.page = ctx, nodes, page
        tab, pages = a_table(ctx, page, seed)
        g = torch.Generator().manual_seed(seed + 1)
        codes = torch.randint(-127, 128, (pages, Hkv, 2, D), generator=g, dtype=torch.int8).sort(2, descending=True).values
        exps = torch.randint(118, 122, (pages, Hkv), generator=g, dtype=torch.uint8)
        self.index, self.tab = mx.PageIndex(codes.to(d), exps.to(d), page), tab.to(d)
        self.q = randn(seed + 2, sum(nodes), Hq, D, scale=1.5).to(d)
        self.cu = ints([0] + torch.tensor(nodes).cumsum(0).tolist())
        self.len = ints(ctx)

    def run(self, n_sel, **kw):
        return mx.attn_select(self.q, self.cu, self.index, self.tab, self.len, n_sel, **kw)

    def check(self, out, n_sel, what, first=1, last=1):
        want = long_ref.select(self.q, self.nodes, self.index.codes, self.index.exps, self.tab, self.ctx, self.page, n_sel,
                               first, last, self.q.shape[0])
        seen = want[:, 0, 0] != -7
        got = out.cpu()
        assert torch.equal(got[seen], want[seen]), f"{what}: first at {(got[seen] != want[seen]).nonzero()[0].tolist()}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,nodes,Hq,Hkv,page,n_sel,first,last", [
    ([0], [1], 4, 1, 16, 4, 1, 1), ([1], [2], 4, 4, 16, 1, 0, 1), ([100], [1], 8, 1, 16, 7, 1, 1), ([113], [1], 8, 1, 16, 7, 1, 1),
    ([1000, 17, 0, 640], [8, 8, 8, 8], 16, 2, 16, 12, 1, 2), ([4096], [64], 32, 2, 64, 9, 0, 3), ([3000, 900], [5, 1], 71, 1, 32, 5, 2, 1),
    ([2000], [2], 128, 1, 16, 30, 10, 20), ([10000, 1, 9999], [3, 4, 2], 12, 4, 32, 64, 1, 2), ([16000], [1], 64, 8, 256, 16, 1, 1),
    ([40000], [1], 10, 2, 16, 512, 1, 1),
])
def test_select(D, ctx, nodes, Hq, Hkv, page, n_sel, first, last):
    c = Select(ctx, nodes, Hq, Hkv, D, page, seed=sum(ctx) + Hq)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    c.check(c.run(n_sel, first=first, last=last, dev_status=status), n_sel, f"{ctx} {nodes} {Hq}/{Hkv} D={D} page={page}", first, last)
    assert mx.mxg_query_status(status) == 0


def test_select_many_sequences():
    g = torch.Generator().manual_seed(7)
    ctx = torch.randint(0, 500, (260,), generator=g).tolist()
    nodes = torch.randint(0, 3, (260,), generator=g).tolist()
    c = Select(ctx, nodes, 4, 2, 64, 16, seed=3)
    c.check(c.run(6), 6, "many")


def test_select_long():
    c = Select([200001], [2], 4, 2, 64, 16, seed=5)
    c.check(c.run(33), 33, "long")
    c = Select([16 * 32768], [1], 2, 1, 128, 16, seed=6)  # the longest table
    c.check(c.run(70), 70, "longest")


def test_select_equal_scores():
    """Equal scores go to the lowest page; scores that differ by one in 2^20 do not count as equal."""
    c = Select([3200], [3], 8, 2, 128, 16, seed=9)
    codes = c.index.codes
    codes[:] = codes[0]
    c.index.exps[:] = 120
    c.check(c.run(9), 9, "all equal")
    codes[c.tab[0, 77].long(), :, 0] += 1
    codes[c.tab[0, 123].long(), :, 1] -= 1
    codes.clamp_(-127, 127)
    c.check(c.run(9), 9, "two above")
    codes[:] = torch.tensor([[127] * 128, [-127] * 128])
    c.q[:] = 127.0
    codes[c.tab[0, 150].long(), :, 0, 0] = 126
    codes[c.tab[0, 1].long(), :, 0, 0] = 126
    c.check(c.run(198), 198, "the two that are one step below")
    c.index.exps[c.tab[0, 50:150].long()] = 119  # half
    c.q[1] *= -1
    c.q[2] = 0
    c.check(c.run(101), 101, "halves")
    codes[:] = 0
    c.check(c.run(101), 101, "zeros")


def test_select_of_every_magnitude():
    c = Select([1600], [9], 8, 2, 64, 16, seed=10)
    c.index.exps[:] = torch.randint(27, 250, c.index.exps.shape, generator=torch.Generator().manual_seed(1), dtype=torch.uint8).to(dev())
    for i, s in enumerate([0.0, 1e-38, 2.0 ** -110, 1e-30, 1e30, 8e36]):
        c.q[i] *= s
    c.q[6, 0, 3], c.q[7, 5, 1] = float("nan"), float("-inf")  # the kv head counts as zero, the other one does not
    c.check(c.run(20), 20, "magnitudes")
    c.index.exps[c.tab[0, 40].long()] = 255
    c.index.exps[c.tab[0, 60].long(), 1] = 255
    out = c.run(20)
    assert bool((out == 40).any(-1).all()) and bool((out[:, 1] == 60).any(-1).all())
    c.check(out, 20, "without bounds")


def test_select_ranges_and_padding():
    c = Select([800, 333], [4, 3], 8, 2, 64, 16, seed=11)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    c.tab[0, 3], c.tab[0, 20], c.tab[0, 0] = -9, 1 << 30, -1  # (the first page is taken without its bounds)
    c.check(c.run(10, dev_status=status), 10, "pages outside")
    assert mx.mxg_query_status(status) == 5
    c = Select([800, 333], [4, 3], 8, 2, 64, 16, seed=11)
    c.q = torch.cat([c.q, torch.full((5, 8, 64), float("nan"), dtype=torch.bfloat16, device=dev())])
    out = torch.full((12, 2, 10), 99, dtype=torch.int32, device=dev())
    c.run(10, out=out, dev_status=status)
    assert mx.mxg_query_status(status) == 0 and bool((out[7:] == 99).all())
    c.check(out, 10, "padded batch")
    c.len = ints([800, 100000])  # as many as the table has
    c.ctx = [800, c.tab.shape[1] * 16]
    c.run(10, out=out, dev_status=status)
    assert mx.mxg_query_status(status) == 5
    c.cu, c.nodes = ints([0, 4, 99]), [4, 8]
    c.q = c.q.nan_to_num()
    c.len, c.ctx = ints([800, 333]), [800, 333]
    c.check(c.run(10, dev_status=status), 10, "offsets")
    assert mx.mxg_query_status(status) == 5


def test_select_strides_stream_and_repeats():
    c = Select([5000, 2000], [8, 64], 12, 4, 128, 32, seed=13)
    want = c.run(21, last=2)
    c.check(want, 21, "plain", 1, 2)
    wide = torch.cat([c.q, c.q], 1)
    c.q = wide[:, 12:]
    big = torch.zeros(c.index.codes.shape[0], 4, 3, 256, dtype=torch.int8, device=dev())
    big[:, :, 1] = c.index.codes.flatten(-2)
    c.index = mx.PageIndex(big[:, :, 1].unflatten(-1, (2, 128)), c.index.exps, 32)
    for _ in range(3):
        assert torch.equal(c.run(21, last=2), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.run(21, last=2, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("Hq,Hkv,D", [(64, 8, 128), (10, 2, 64), (3, 1, 128), (24, 8, 64), (128, 1, 128), (4, 4, 64), (40, 4, 128)])
def test_select_of_wide_trees(Hq, Hkv, D):
    """Trees of up to 64 nodes beside single ones: several passes, one after another or beside one another, rows that need
    no choice among them."""
    ctx, nodes = [3339, 0, 760, 5134, 46, 12001, 330, 815], [64, 33, 1, 20, 30, 2, 1, 41]
    for times in (1, 4):
        c = Select(ctx * times, nodes * times, Hq, Hkv, D, 32, seed=Hq + times)
        c.check(c.run(11, first=2, last=3), 11, f"{times}", 2, 3)

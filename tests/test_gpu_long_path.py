"""The long-context operators as they are used: a step over selected pages after prompts, by itself, in a CUDA graph and
beside others; the example."""
import os
import sys

import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
import test_gpu_attn_shared as shared
import test_gpu_attn_sparse as sparse
from gpu_util import dev

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Step:
    """Two layers, sequences of ctx tokens in the cache with their bounds, a tree each."""

    def __init__(self, ctx, nodes, n_sel, Hq=16, Hkv=2, D=128, page=32, room=16):
        d = dev()
        self.case = sparse.Case(ctx, nodes, Hq, Hkv, D, page, n_sel, seed=31)
        c = self.case
        self.n_sel, self.page = n_sel, page
        need = [-(-(x + room) // page) for x in ctx]
        order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(1)).tolist()
        tab = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            tab[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        self.tab = tab.to(d)
        shape = (2, sum(need) + 2, page, Hkv, D)
        g = torch.Generator().manual_seed(2)
        self.cache = mx.KVCache(torch.randn(*shape, generator=g).bfloat16().to(d), torch.randn(*shape, generator=g).bfloat16().to(d))
        self.index = mx.PageIndex.of(self.cache)
        mx.kv_index(self.cache, self.index, self.tab, None, c.len)
        self.accept = torch.tensor([[0, n - 1] if n > 1 else [0, -1] for n in nodes], dtype=torch.int32, device=d)
        self.sel = [torch.empty(sum(nodes), Hkv, n_sel, dtype=torch.int32, device=d) for _ in range(2)]
        self.out = [torch.empty_like(c.q) for _ in range(2)]
        self.ctx_out = torch.empty_like(c.len)

    def run(self, stream=None):
        c, kw = self.case, dict(stream=stream)
        for i in range(2):
            mx.attn_select(c.q, c.cu, self.index.layer(i), self.tab, c.len, self.n_sel, out=self.sel[i], **kw)
            mx.attn_sparse(c.q, c.k, c.v, c.cu, c.mask, self.cache.layer(i), self.tab, c.len, self.sel[i], out=self.out[i], **kw)
        ks, vs = torch.stack([c.k, c.k * 2]), torch.stack([c.v, c.v * 2])
        mx.kv_append(ks, vs, c.cu, self.accept, self.cache, self.tab, c.len, ctx_out=self.ctx_out, **kw)
        mx.kv_index(self.cache, self.index, self.tab, c.len, self.ctx_out, **kw)

    def check(self, what):
        import long_ref
        c = self.case
        for i in range(2):
            x = self.index.layer(i)
            want = long_ref.select(c.q, c.nodes, x.codes, x.exps, self.tab, c.ctx, self.page, self.n_sel, 1, 1, c.q.shape[0])
            assert torch.equal(self.sel[i].cpu(), want), f"{what}: pages of layer {i}"
            l = self.cache.layer(i)
            for at, o, b in long_ref.sparse(c.q, c.k, c.v, c.nodes, c.mask, l.k, l.v, self.tab, c.ctx, self.sel[i], c.scale):
                long_ref.assert_within(self.out[i][at], o, b, f"{what}: layer {i}")
        full = set()
        for b, n in enumerate(self.ctx_out.tolist()):
            full |= {int(self.tab[b, j]) for j in range(n // self.page)}
        for pg in full:
            for i in range(2):
                for h in range(c.k.shape[1]):
                    codes, code = long_ref.bounds(self.cache.k[i, pg, :, h])
                    assert int(self.index.exps[i, pg, h]) == code and torch.equal(self.index.codes[i, pg, h].cpu(), codes), (what, pg)


def test_step():
    s = Step([700, 31, 63, 0, 412], [3, 2, 1, 1, 8], 7)
    s.run()
    s.check("a step")
    assert s.ctx_out.tolist() == [702, 33, 64, 1, 414]


def test_step_in_a_graph():
    """Captured once, replayed with other values in the same tensors."""
    s = Step([700, 31, 63, 0, 412], [3, 2, 1, 1, 8], 7)
    s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        s.run()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            s.run()
    gen = torch.Generator().manual_seed(5)
    s.case.q.copy_(torch.randn(*s.case.q.shape, generator=gen).bfloat16() * 2)
    s.case.k.copy_(torch.randn(*s.case.k.shape, generator=gen).bfloat16())
    for x in s.sel:
        x.fill_(-9)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    s.check("replayed")


def test_two_graphs_and_two_streams():
    """Two captured graphs, and eager calls on two streams at once, do not share what they write."""
    a, b = Step([900, 200], [4, 1], 6), Step([64, 1500, 300], [1, 8, 2], 9)
    c = shared.Case([2], [512], [100, 300, 40], [8, 1, 3], 16, 2, 128, 64, seed=4)
    want = c.run()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, st in zip((a, b), streams):
        with torch.cuda.stream(st):
            s.run()
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                s.run()
            graphs.append(g)
    got = []
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                got.append(c.run())
    torch.cuda.synchronize()
    a.check("first graph")
    b.check("second graph")
    assert all(torch.equal(x, want) for x in got)


def test_shared_in_a_graph():
    c = shared.Case([3, 2], [640, 128], [100, 0, 7, 300, 64], [1, 8, 2, 1, 4], 16, 2, 128, 64, seed=6)
    out = torch.empty_like(c.q)
    c.run(out=out)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(out=out)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            c.run(out=out)
    c.q.mul_(-1.5)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check(out, "replayed")


def test_results_in_place_of_q():
    for module, args in ((shared, ([2], [512], [100, 300, 40], [8, 1, 3], 16, 2, 128, 64)),
                         (sparse, ([900, 200, 0], [8, 1, 3], 16, 2, 64, 32, 5))):
        c = module.Case(*args, seed=8)
        want = c.run()
        q = c.q
        assert c.run(out=q) is not None and torch.equal(q, want)


def test_example():
    import attention_step
    got, want = attention_step.run_long(512, 4, 2, 128, (700, 45, 1024), device=dev())
    assert got.shape == want.shape
    off = float((got.double() - want.double()).norm() / want.double().norm())
    assert off < 2.0 ** -6, off


def test_offsets_past_32_bits():
    """The same keys in a cache of 5 GB, past 2^31 elements from its beginning: the same bits."""
    page, hkv, d, far = 64, 8, 128, 40000
    g = torch.Generator(device="cuda").manual_seed(50)
    small = torch.randn(12, page, hkv, d, generator=g, device="cuda").bfloat16()
    big = torch.empty(far + 12, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    big[far:] = small
    q = torch.randn(3, 16, d, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(3, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, ctx, mask = ints([0, 1, 3]), ints([350, 300]), torch.tensor([1, 1, 3], device="cuda")
    outs = []
    for pages, base in ((small, 0), (big, far)):
        tab = ints([[0, 1, 2, 3, 4, 5], [0, 1, 8, 9, 10, 11]]) + base
        cache = mx.KVCache(pages, pages)
        index = mx.kv_index(cache, mx.PageIndex.of(cache), tab, None, ctx)
        sel = mx.attn_select(q, cu, index, tab, ctx, 4)
        outs.append([index.codes[base:], index.exps[base:], sel,
                     mx.attn_sparse(q, k, v, cu, mask, cache, tab, ctx, sel),
                     mx.attn_shared(q, k, v, cu, mask, cache, tab, ctx, ints([0, 2]), ints([128]))])
    for a, b in zip(*outs):
        assert torch.equal(a, b)

"""Long contexts, held to the relative length of each row's error: a result
shrinks with the number of keys, so that a bound of each value by the size of v
no longer sees a tile of keys that is left out."""
import math

import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev
from test_gpu_attn_prompt import inputs, offsets
from test_gpu_attn_tree import Case

pytestmark = pytest.mark.gpu

# The rounding of the result moves each value by at most 2^-8 of itself, and so
# the row by at most 2^-8 of its length.  Those of the weights, at most 2^-8 of
# each and independent, move it by 2^-8 sqrt(sum p^2 v^2) in the root mean
# square, which for independent values v is the row's own length.  Both
# together: 2^-7.  A tile of 128 keys left out of n moves the row by about
# sqrt(128 / n) of its length, 0.056 at 40001.
LIMIT = 2.0 ** -7


def softmax_rows(q, k, v, see, scale):
    """64 bits: q (M, D), k, v (K, D), see (M, K) -> (M, D)."""
    s = (q.double() @ k.double().T * scale).masked_fill(~see, -math.inf)
    return torch.softmax(s, 1) @ v.double()


def off(got, want):
    return float(((got.double() - want).norm(dim=1) / want.norm(dim=1)).max())


def cached(c, b, h):
    """k and v of sequence b's cached tokens and nodes, kv head h."""
    j = torch.arange(c.ctx[b], device=c.q.device)
    page = c.kc.shape[1]
    pg, a = c.tab[b].long()[j // page], sum(c.nodes[:b])
    n = c.nodes[b]
    return (torch.cat([c.kc[pg, j % page, h], c.k[a:a + n, h]]), torch.cat([c.vc[pg, j % page, h], c.v[a:a + n, h]]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,nodes,page", [([40001, 100], [3, 2], 64), ([4000], [1], 16), ([9001, 0, 2500], [8, 3, 64], 256),
                                            ([32768, 5], [1, 1], 128)])
def test_tree_long_contexts(D, ctx, nodes, page):
    Hq, Hkv = 4, 2
    c = Case(ctx, nodes, Hq, Hkv, D, page, seed=40 + D)
    out = c.run()
    a = 0
    for b, n in enumerate(nodes):
        for h in range(Hq):
            k, v = cached(c, b, h // (Hq // Hkv))
            new = (c.mask[a:a + n, None] >> torch.arange(n, device=out.device) & 1).bool()
            see = torch.cat([torch.ones(n, ctx[b], dtype=torch.bool, device=out.device), new], 1)
            want = softmax_rows(c.q[a:a + n, h], k, v, see, c.scale)
            assert off(out[a:a + n, h], want) < LIMIT, (b, h)
        a += n


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_long_rows(D):
    d = dev()
    lens, Hq, Hkv = [9000, 130], 4, 2
    q, k, v = inputs(41, sum(lens), Hq, Hkv, D, d)
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    rows = torch.cat([torch.arange(300, 9000, 83), torch.tensor([8959, 8960, 8998, 8999])]).to(d)
    see = torch.arange(9000, device=d) <= rows[:, None]
    for h in range(Hq):
        want = softmax_rows(q[rows, h], k[:9000, h // 2], v[:9000, h // 2], see, D ** -0.5)
        assert off(out[rows, h], want) < LIMIT, h

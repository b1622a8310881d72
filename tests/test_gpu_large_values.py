"""attn_shared and attn_sparse with values near fp32's largest, where a row's first key counts for 2^-28 of the others: with
that key as the row's reference the sums pass 2^128, with the maximum they do not."""
import pytest
import torch

import test_gpu_attn_shared as shared
import test_gpu_attn_sparse as sparse

pytestmark = pytest.mark.gpu


def low_first_keys(c, tokens, value):
    """Channel 0 gives the keys at `tokens` of every sequence scores 28 ln 2 below the others, which differ by little."""
    D = c.q.shape[-1]
    c.q *= 0.05
    c.q[..., 0] = 4.0
    c.kc[..., 0], c.k[..., 0] = 0.0, 0.0
    low = -28 * 0.6931471805599453 / (4.0 * c.scale)
    for b in range(c.tab.shape[0]):
        for t in tokens(b):
            page = int(c.tab[b, t // c.kc.shape[1]])
            if page >= 0:
                c.kc[page, t % c.kc.shape[1], :, 0] = low
    c.v, c.vc = c.v * value, c.vc * value
    assert D in (64, 128)


@pytest.mark.parametrize("value", [2.0**76, 2.0**98, 2.0**108])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes", [[1, 1], [4, 2], [8, 5], [16, 3]])
def test_sparse(nodes, D, value):
    c = sparse.Case([900, 333], nodes, 8, 2, D, 64, 9, seed=23)
    c.sel[:, :, 0] = 0
    low_first_keys(c, lambda b: [0], value)
    c.tab[0, 3] = -4  # a page outside the cache: keys and values of zero
    out = c.run()
    assert bool(torch.isfinite(out.float()).all())
    c.check(out, f"{nodes} {value}")


@pytest.mark.parametrize("value", [2.0**76, 2.0**98, 2.0**108])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nodes,Hq,Hkv", [(1, 8, 4), (4, 16, 4), (8, 8, 4)])
def test_shared(nodes, Hq, Hkv, D, value):
    c = shared.Case([48], [256], [7 * i % 300 for i in range(48)], [nodes] * 48, Hq, Hkv, D, 64, seed=24)
    low_first_keys(c, lambda b: [0, 256] if c.ctx[b] > 256 else [0], value)
    out = c.run()
    assert bool(torch.isfinite(out.float()).all())
    c.check(out, f"{nodes} {Hq}/{Hkv} {value}")

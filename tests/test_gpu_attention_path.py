"""The attention operators together, as examples/attention_step.py runs them:
prompt pass into the cache, verified tree, accepted path, next token."""
import os
import sys

import pytest
import torch

from gpu_util import dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,hq,hkv,d,lens", [(512, 4, 2, 128, (300, 45, 1)), (1024, 16, 2, 64, (64, 500)),
                                                  (7168, 64, 8, 128, (130, 7))])
def test_cache_path_is_the_prompt(hidden, hq, hkv, d, lens):
    """The token after an accepted path attends to the cache as it would to the
    same tokens in one prompt.  q, k and v come from GEMMs of other shapes, whose
    fp32 sums may round to the neighbouring bf16 value (2^-8) here and there;
    the softmax weights and the result are rounded to bf16 once each: 2^-6 of
    the norm holds all of them."""
    dev()
    import attention_step
    got, want = attention_step.run(hidden, hq, hkv, d, lens)
    assert got.shape == (len(lens), hq, d)
    off = (got.float() - want.float()).norm(dim=(1, 2)) / want.float().norm(dim=(1, 2))
    assert float(off.max()) < 2.0 ** -6, off


def test_steps_in_a_graph():
    """The operators of a verify step can be captured and replayed, on inputs
    that change between replays."""
    d = dev()
    import attention_step
    import fp8_block_scaled_dynamic_gb300 as mx
    from test_gpu_attn_tree import Case
    c = Case([700, 90], [5, 3], 16, 2, 128, 64, seed=4)
    cs = attention_step.rope_table(64, 128, d)
    pos = torch.arange(8, device=d).int()
    q0, k0 = c.q.clone(), c.k.clone()
    cache = mx.KVCache(c.kc, c.vc)
    out, qo, ko = torch.empty_like(c.q), torch.empty_like(c.q), torch.empty_like(c.k)

    def step():
        mx.qk_norm_rope(q0, k0, pos, cs, q_out=qo, k_out=ko)
        mx.attn_tree(qo, ko, c.v, c.cu, c.mask, cache, c.tab, c.len, out=out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        q0.copy_(c.q * (1 + i))
        g.replay()
        again = out.clone()
        step()
        assert torch.equal(out, again)
    c.q, c.k = qo, ko
    c.check(out, "replayed")

"""What the attention entry points refuse before anything is launched."""
import ctypes

import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from fp8_block_scaled_dynamic_gb300.attention import AttnOpts, CacheDesc, Heads

P = 1 << 20  # a 16-byte aligned pointer value; nothing is dereferenced on these paths


def H(ptr=P, tok=1024, head=128):
    return Heads(ptr, tok, head)


def C(**kw):
    f = dict(k=P, v=P, layer_stride=0, page_stride=1 << 16, slot_stride=1024, head_stride=128, layers=1, pages=4, page_size=64)
    f.update(kw)
    return CacheDesc(**f)


ROPE = dict(q=H(), k=H(), T=4, Hq=8, Hkv=2, D=128, wq=P, wk=P, eps=1e-6, pos=P, cs=P, max_pos=64, rot=128, inter=0, qo=H(),
            ko=H(), v=None, cache=None, slots=None, status=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(D=0), 1), (dict(D=20, rot=0), 2), (dict(D=8, rot=0), 2), (dict(D=264, rot=0), 2), (dict(rot=8), 2),
    (dict(rot=144), 1), (dict(rot=-16), 1), (dict(inter=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(cs=None), 1), (dict(pos=None), 1), (dict(max_pos=0), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(ko=None), 1),
    (dict(q=H(ptr=P + 2)), 3), (dict(q=H(tok=1020)), 3), (dict(k=H(head=-8)), 1), (dict(k=H(tok=1 << 40)), 3),
    (dict(wq=P + 8), 3), (dict(cs=P + 4), 3), (dict(pos=P + 2), 3), (dict(status=P + 1), 3),
    (dict(cache=C()), 1), (dict(cache=C(), slots=P), 1), (dict(cache=C(page_size=48), slots=P, v=H()), 2),
    (dict(cache=C(k=None), slots=P, v=H()), 1), (dict(cache=C(pages=0), slots=P, v=H()), 1),
    (dict(cache=C(slot_stride=4), slots=P, v=H()), 3), (dict(cache=C(), slots=P + 4, v=H()), 3),
])
def test_rope_refusals(kw, want):
    a = {**ROPE, **kw}
    assert mx.lib().qk_norm_rope(*a.values()) == want


PROMPT = dict(q=H(), k=H(), v=H(), cu=P, B=2, T=10, Hq=8, Hkv=2, D=128, scale=0.1, out=H(), opts=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(cu=None), 1), (dict(scale=float("inf")), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(Hkv=3), 2), (dict(D=96), 2), (dict(Hq=258, Hkv=2), 2), (dict(B=4097), 2), (dict(q=None), 1), (dict(out=H(ptr=None)), 1),
    (dict(v=H(ptr=P + 8)), 3), (dict(k=H(tok=4)), 3), (dict(cu=P + 1), 3), (dict(opts=AttnOpts(debug_stall=2)), 1),
    (dict(opts=AttnOpts(dev_status=P + 2)), 3), (dict(k=H(head=0)), 2), (dict(q=H(tok=0)), 2),
])
def test_prompt_refusals(kw, want):
    assert mx.lib().attn_prompt(*{**PROMPT, **kw}.values()) == want


TREE = dict(q=H(), k=H(), v=H(), cu=P, mask=P, B=2, N=10, cache=C(), table=P, ld=8, cols=8, ctx=P, Hq=8, Hkv=2, D=128, scale=0.1,
            out=H(), opts=AttnOpts(P, 1 << 40), stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(N=-1), 1), (dict(mask=None), 1), (dict(ctx=None), 1), (dict(cache=None), 1), (dict(table=None), 1),
    (dict(ld=7), 1), (dict(cols=-1), 1), (dict(cache=C(page_size=8)), 2), (dict(cache=C(page_size=512)), 2), (dict(D=32), 2),
    (dict(Hkv=3), 2), (dict(cols=1 << 25, ld=1 << 25), 2), (dict(mask=P + 4), 3), (dict(cache=C(v=P + 8)), 3),
    (dict(cache=C(head_stride=12)), 3), (dict(table=P + 2), 3), (dict(cache=C(page_stride=0)), 2), (dict(cache=C(head_stride=0)), 2),
])
def test_tree_refusals(kw, want):
    assert mx.lib().attn_tree(*{**TREE, **kw}.values()) == want


APPEND = dict(k=H(), kl=0, v=H(), vl=0, cu=P, B=2, N=10, accept=P, lda=4, most=4, cache=C(), table=P, ld=8, cols=8, ctx=P, Hkv=2,
              D=128, ctx_out=P + 64, status=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(N=-1), 1), (dict(cu=None), 1), (dict(accept=None), 1), (dict(lda=3), 1), (dict(ctx=None), 1),
    (dict(ctx_out=P), 1), (dict(ld=2), 1), (dict(cache=None), 1), (dict(kl=-8), 1), (dict(kl=4), 3), (dict(D=12), 2),
    (dict(D=2048), 2), (dict(B=5000), 2), (dict(cache=C(layers=0)), 1), (dict(cache=C(layers=70000)), 2), (dict(k=None), 1),
    (dict(v=H(ptr=P + 4)), 3), (dict(accept=P + 1), 3),
])
def test_append_refusals(kw, want):
    assert mx.lib().kv_append(*{**APPEND, **kw}.values()) == want


def test_workspace_query_of_a_head_width_it_has_not():
    assert mx.mxg_attn_tree_workspace_bytes(96) == 0


def test_binding_checks_tensors():
    """CPU tensors, other types and shapes that do not fit raise ValueError."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.attn_prompt(x, x, x, cu)
    with pytest.raises(ValueError):
        mx.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        mx.KVCache(x, x)

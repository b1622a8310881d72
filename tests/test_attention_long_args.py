"""What the long-context entry points refuse before anything is launched."""
import pytest

import fp8_block_scaled_dynamic_gb300 as mx
from fp8_block_scaled_dynamic_gb300.attention import AttnOpts, IndexDesc
from test_attention_args import C, H, P


def X(**kw):
    f = dict(codes=P, exps=P, codes_layer=0, codes_page=2048, codes_head=256, exps_layer=0, exps_page=8, layers=1, pages=4)
    f.update(kw)
    return IndexDesc(**f)


PAGED = [
    (dict(B=0), 1), (dict(N=-1), 1), (dict(mask=None), 1), (dict(ctx=None), 1), (dict(cache=None), 1), (dict(table=None), 1),
    (dict(cu=None), 1), (dict(cols=9), 1), (dict(cols=-1), 1), (dict(Hkv=3), 2), (dict(D=96), 2), (dict(B=4097), 2),
    (dict(Hq=258), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(q=H(ptr=P + 2)), 3), (dict(out=None), 1),
    (dict(v=H(tok=0)), 2), (dict(cache=C(page_size=8)), 2), (dict(cache=C(page_stride=0)), 2), (dict(mask=P + 4), 3),
    (dict(ctx=P + 2), 3), (dict(table=P + 1), 3), (dict(opts=AttnOpts(P, 1 << 40, debug_stall=2)), 1),
    (dict(cols=1 << 27, ld=1 << 27), 2), (dict(opts=AttnOpts(P, 1 << 40, P + 2)), 3),
]
SHARED = dict(q=H(), k=H(), v=H(), cu=P, mask=P, B=2, N=10, cache=C(), table=P, ld=8, cols=8, ctx=P, groups=P, prefix=P, n_groups=1,
              Hq=8, Hkv=2, D=128, scale=0.1, out=H(), opts=AttnOpts(P, 1 << 40), stream=None)


@pytest.mark.parametrize("kw,want", PAGED + [
    (dict(n_groups=-1), 1), (dict(n_groups=3), 1), (dict(groups=None), 1), (dict(prefix=None), 1), (dict(groups=P + 2), 3),
    (dict(prefix=P + 1), 3),
])
def test_shared_refusals(kw, want):
    assert mx.lib().attn_shared(*{**SHARED, **kw}.values()) == want


SPARSE = dict(q=H(), k=H(), v=H(), cu=P, mask=P, B=2, N=10, cache=C(), table=P, ld=8, cols=8, ctx=P, sel=P, n_sel=4, Hq=8, Hkv=2,
              D=128, scale=0.1, out=H(), opts=AttnOpts(P, 1 << 40), stream=None)


@pytest.mark.parametrize("kw,want", PAGED + [
    (dict(sel=None), 1), (dict(n_sel=0), 1), (dict(n_sel=513), 2), (dict(sel=P + 2), 3), (dict(cols=1 << 20, ld=1 << 20), 2),
])
def test_sparse_refusals(kw, want):
    assert mx.lib().attn_sparse(*{**SPARSE, **kw}.values()) == want


SELECT = dict(q=H(), cu=P, B=2, N=10, index=X(), page=64, table=P, ld=8, cols=8, ctx=P, Hq=8, Hkv=2, D=128, n_sel=4, first=1, last=1,
              sel=P, status=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(N=-1), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(index=None), 1), (dict(table=None), 1), (dict(sel=None), 1),
    (dict(cols=9), 1), (dict(n_sel=0), 1), (dict(first=-1), 1), (dict(last=0), 1), (dict(first=4), 1), (dict(last=4), 1), (dict(last=2147483647), 1),
    (dict(page=0), 1), (dict(page=24), 2), (dict(n_sel=513), 2), (dict(D=96), 2), (dict(Hkv=3), 2), (dict(Hq=258), 2), (dict(B=4097), 2),
    (dict(q=None), 1), (dict(q=H(tok=4)), 3), (dict(sel=P + 2), 3), (dict(cu=P + 2), 3), (dict(ctx=P + 1), 3),
    (dict(status=P + 1), 3), (dict(cols=32769, ld=32769), 2),
    (dict(index=X(codes=None)), 1), (dict(index=X(exps=None)), 1), (dict(index=X(pages=0)), 1), (dict(index=X(layers=0)), 1),
    (dict(index=X(codes=P + 8)), 3), (dict(index=X(codes_page=8)), 3), (dict(index=X(codes_head=-16)), 1), (dict(index=X(exps_page=-1)), 1),
    (dict(index=X(codes_head=1 << 39)), 3), (dict(index=X(codes_page=1 << 31)), 3), (dict(index=X(exps_page=1 << 31)), 3),
    (dict(cols=1 << 27, ld=1 << 27), 2),
])
def test_select_refusals(kw, want):
    assert mx.lib().attn_select(*{**SELECT, **kw}.values()) == want


INDEX = dict(cache=C(), Hkv=2, D=128, index=X(), table=P, B=2, ld=8, cols=8, old=P, now=P, status=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(now=None), 1), (dict(cols=9), 1), (dict(table=None), 1), (dict(cache=None), 1),
    (dict(index=None), 1), (dict(D=96), 2), (dict(B=4097), 2), (dict(Hkv=65536), 2), (dict(index=X(pages=3)), 1), (dict(cache=C(layers=2)), 1),
    (dict(cache=C(page_size=20)), 2), (dict(cols=1 << 26, ld=1 << 26), 2), (dict(now=P + 2), 3), (dict(old=P + 1), 3), (dict(table=P + 2), 3),
    (dict(status=P + 2), 3), (dict(index=X(codes=P + 4)), 3), (dict(cols=1 << 24, ld=1 << 24, B=200), 2),
    (dict(index=X(codes_page=0)), 2), (dict(index=X(codes_head=128)), 2), (dict(index=X(exps_page=1)), 2),
    (dict(index=X(layers=2)), 2), (dict(index=X(layers=2, codes_layer=8192)), 2),
])
def test_index_refusals(kw, want):
    assert mx.lib().kv_index(*{**INDEX, **kw}.values()) == want


def test_workspace_sizes_of_nothing():
    L = mx.lib()
    assert L.mxg_attn_shared_workspace_bytes(4, 8, 96) == 0 and L.mxg_attn_shared_workspace_bytes(-1, 8, 128) == 0
    assert L.mxg_attn_sparse_workspace_bytes(4, 2, 0, 128) == 0 and L.mxg_attn_sparse_workspace_bytes(4, 2, 4, 32) == 0

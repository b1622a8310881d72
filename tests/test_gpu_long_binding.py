"""The binding of the long-context operators refuses a tensor that does not fit, before anything is launched."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev

pytestmark = pytest.mark.gpu

N, B, HQ, HKV, D, PAGE, PAGES, SEL = 6, 2, 4, 2, 64, 16, 6, 3


def arguments():
    d = dev()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=d)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=d)  # noqa: E731
    return dict(q=z(N, HQ, D), k=z(N, HKV, D), v=z(N, HKV, D), cu=i32([0, 3, 6]), mask=torch.ones(N, dtype=torch.int64, device=d),
                kc=z(PAGES, PAGE, HKV, D), vc=z(PAGES, PAGE, HKV, D), table=i32([[0, 1, 2], [3, 4, 5]]), ctx=i32([40, 33]),
                groups=i32([0, 2]), prefix=i32([16]), sel=torch.zeros(N, HKV, SEL, dtype=torch.int32, device=d),
                codes=z(PAGES, HKV, 2, D, dtype=torch.int8), exps=z(PAGES, HKV, dtype=torch.uint8), page_size=PAGE, n_sel=SEL,
                out=z(N, HQ, D) + 7, pick=torch.full((N, HKV, SEL), 7, dtype=torch.int32, device=d), first=1, last=1,
                status=torch.zeros(1, dtype=torch.int32, device=d))


def call(op, a):
    if op == "shared":
        return mx.attn_shared(a["q"], a["k"], a["v"], a["cu"], a["mask"], mx.KVCache(a["kc"], a["vc"]), a["table"], a["ctx"],
                              a["groups"], a["prefix"], out=a["out"], dev_status=a["status"], ws=a.get("ws"))
    if op == "sparse":
        return mx.attn_sparse(a["q"], a["k"], a["v"], a["cu"], a["mask"], mx.KVCache(a["kc"], a["vc"]), a["table"], a["ctx"],
                              a["sel"], out=a["out"], dev_status=a["status"], ws=a.get("ws"))
    if op == "select":
        return mx.attn_select(a["q"], a["cu"], mx.PageIndex(a["codes"], a["exps"], a["page_size"]), a["table"], a["ctx"],
                              a["n_sel"], first=a["first"], last=a["last"], out=a["pick"], dev_status=a["status"])
    return mx.kv_index(mx.KVCache(a["kc"], a["vc"]), mx.PageIndex(a["codes"], a["exps"], a["page_size"]), a["table"], a.get("old"),
                       a["ctx"], dev_status=a["status"])


BAD = [
    ("shared sparse", "q", lambda t: t.half()), ("shared sparse", "q", lambda t: t[:5]), ("shared sparse", "k", lambda t: t[..., :32]),
    ("shared sparse", "v", lambda t: t[:, :1]), ("shared sparse", "cu", lambda t: t[:2]), ("shared sparse", "cu", lambda t: t.long()),
    ("shared sparse", "mask", lambda t: t.int()), ("shared sparse", "mask", lambda t: t[:5]), ("shared sparse", "table", lambda t: t[:1]),
    ("shared sparse", "ctx", lambda t: t.cpu()), ("shared sparse", "out", lambda t: t[:, :2]), ("shared sparse", "kc", lambda t: t[:, :, :1]),
    ("shared sparse", "ws", lambda t: torch.zeros(256, dtype=torch.uint8, device="cuda")), ("shared sparse", "status", lambda t: t.long()),
    ("shared", "groups", lambda t: t[:1]), ("shared", "groups", lambda t: t.long()), ("shared", "prefix", lambda t: t.cpu()),
    ("shared", "prefix", lambda t: t.repeat(2)), ("sparse", "sel", lambda t: t[:5]), ("sparse", "sel", lambda t: t.transpose(0, 1)),
    ("sparse", "sel", lambda t: t.long()), ("sparse", "sel", lambda t: t[..., ::2]), ("sparse", "sel", lambda t: t[..., :0]),
    ("select", "q", lambda t: t.half()), ("select", "q", lambda t: t[..., :32]), ("select", "cu", lambda t: t[:2]),
    ("select", "codes", lambda t: t.float()), ("select", "codes", lambda t: t[:, :, :1]), ("select", "codes", lambda t: t[..., :32]),
    ("select", "exps", lambda t: t[:, :1]), ("select", "exps", lambda t: t.int()), ("select", "exps", lambda t: t.cpu()),
    ("select", "page_size", lambda t: 20), ("select", "page_size", lambda t: 1 << 40), ("select", "n_sel", lambda t: 0), ("select", "n_sel", lambda t: 513),
    ("select", "n_sel", lambda t: 2), ("select", "first", lambda t: -1), ("select", "last", lambda t: 0), ("select", "last", lambda t: 3),
    ("select", "pick", lambda t: t[:5]), ("select", "pick", lambda t: t.long()), ("select", "pick", lambda t: t.transpose(0, 1)),
    ("select", "table", lambda t: t[:1]), ("select", "ctx", lambda t: t.long()),
    ("index", "page_size", lambda t: 32), ("index", "codes", lambda t: t[:, :1]), ("index", "codes", lambda t: t[:5]),
    ("index", "exps", lambda t: t[:5]), ("index", "table", lambda t: t[:1]), ("index", "ctx", lambda t: t.long()),
    ("index", "old", lambda t: torch.zeros(3, dtype=torch.int32, device="cuda")), ("index", "kc", lambda t: t[..., ::2]),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refusals(i):
    ops, name, change = BAD[i]
    for op in ops.split():
        a = arguments()
        a[name] = change(a.get(name))
        if name == "kc" and op != "index":
            a["vc"] = a["kc"]
        if name == "kc" and op == "index":
            a["vc"] = a["kc"]
        codes = arguments()["codes"]
        with pytest.raises((ValueError, mx.MxgError)):
            call(op, a)
        torch.cuda.synchronize()
        assert bool((a["out"] == 7).all()) if name != "out" else True
        assert bool((a["pick"] == 7).all()) if name != "pick" else True
        if name != "codes":
            assert torch.equal(a["codes"], codes)


def test_several_layers_are_refused():
    a = arguments()
    layers = mx.KVCache(torch.stack([a["kc"]] * 2), torch.stack([a["vc"]] * 2))
    index = mx.PageIndex.of(layers)
    assert index.codes.shape == (2, PAGES, HKV, 2, D) and index.page_size == PAGE
    with pytest.raises(ValueError):
        mx.attn_select(a["q"], a["cu"], index, a["table"], a["ctx"], SEL)
    with pytest.raises(ValueError):
        mx.attn_sparse(a["q"], a["k"], a["v"], a["cu"], a["mask"], layers, a["table"], a["ctx"], a["sel"])
    with pytest.raises(ValueError):
        mx.attn_shared(a["q"], a["k"], a["v"], a["cu"], a["mask"], layers, a["table"], a["ctx"], a["groups"], a["prefix"])
    with pytest.raises(ValueError):
        mx.kv_index(layers, index.layer(0), a["table"], None, a["ctx"])
    mx.kv_index(layers, index, a["table"], None, a["ctx"])


def test_calls_that_fit():
    for op in ("shared", "sparse", "select", "index"):
        a = arguments()
        call(op, a)
        assert mx.mxg_query_status(a["status"]) == 0


def test_no_nodes():
    a = arguments()
    for n in ("q", "k", "v", "mask", "sel", "out", "pick"):
        a[n] = a[n][:0]
    a["cu"] = torch.zeros(3, dtype=torch.int32, device=dev())
    for op in ("shared", "sparse", "select"):
        assert call(op, a).shape[0] == 0

"""The binding of the attention operators refuses a tensor that does not fit,
before anything is launched: calls that are right but for one argument."""
import pytest
import torch

import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev

pytestmark = pytest.mark.gpu

T, B, HQ, HKV, D, PAGE, PAGES, LAYERS, MOST = 12, 3, 4, 2, 64, 16, 6, 2, 4


def call(op, change):
    """A call that is right but for `change`: the ValueError that it raises, or
    None, and whether all that it may write is as before."""
    d = dev()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=d)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=d)  # noqa: E731
    a = dict(q=z(T, HQ, D), k=z(T, HKV, D), v=z(T, HKV, D), kc=z(PAGES, PAGE, HKV, D), vc=z(PAGES, PAGE, HKV, D),
             cu=i32([0, 4, 8, 12]), table=i32([[0, 1], [2, 3], [4, 5]]), ctx=i32([1, 2, 3]), status=None)
    if op == "rope":
        a.update(pos=i32(range(T)), cos_sin=z(32, D, dtype=torch.float32), wq=z(D), wk=z(D), q_out=z(T, HQ, D) + 7,
                 k_out=z(T, HKV, D) + 7, slots=torch.arange(T, device=d))
    elif op == "append":
        a.update(k=z(LAYERS, T, HKV, D), v=z(LAYERS, T, HKV, D), kc=z(LAYERS, PAGES, PAGE, HKV, D) + 7,
                 vc=z(LAYERS, PAGES, PAGE, HKV, D) + 7, accept=i32([[0, 1, -1, -1]] * B), ctx_out=i32([7] * B))
    else:
        a.update(out=z(T, HQ, D) + 7, mask=torch.ones(T, dtype=torch.int64, device=d),
                 ws=z(mx.mxg_attn_tree_workspace_bytes(D), dtype=torch.uint8))
    a.update({n: f(a[n]) for n, f in change.items()})
    written = [a[n] for n in ("out", "q_out", "k_out", "ctx_out") if torch.is_tensor(a.get(n)) and a[n].is_cuda]
    if op in ("rope", "append"):
        written += [a["kc"], a["vc"]]
    before, error = [w.clone() for w in written], None
    try:
        if op == "rope":
            mx.qk_norm_rope(a["q"], a["k"], a["pos"], a["cos_sin"], wq=a["wq"], wk=a["wk"], q_out=a["q_out"],
                            k_out=a["k_out"], v=a["v"], cache=mx.KVCache(a["kc"], a["vc"]), slots=a["slots"],
                            dev_status=a["status"])
        elif op == "prompt":
            mx.attn_prompt(a["q"], a["k"], a["v"], a["cu"], out=a["out"], dev_status=a["status"])
        elif op == "tree":
            mx.attn_tree(a["q"], a["k"], a["v"], a["cu"], a["mask"], mx.KVCache(a["kc"], a["vc"]), a["table"], a["ctx"],
                         out=a["out"], ws=a["ws"], dev_status=a["status"])
        else:
            mx.kv_append(a["k"], a["v"], a["cu"], a["accept"], mx.KVCache(a["kc"], a["vc"]), a["table"], a["ctx"],
                         ctx_out=a["ctx_out"], dev_status=a["status"])
    except ValueError as e:
        error = e
    torch.cuda.synchronize()
    return error, all(torch.equal(w, b) for w, b in zip(written, before))


@pytest.mark.parametrize("op", ["rope", "prompt", "tree", "append"])
def test_the_call_without_a_fault_is_taken(op):
    assert call(op, {}) == (None, False)


cpu = lambda x: x.cpu()  # noqa: E731
f32 = lambda x: x.float()  # noqa: E731
half = lambda x: x.half()  # noqa: E731
i64 = lambda x: x.long()  # noqa: E731
i32 = lambda x: x.int()  # noqa: E731
short = lambda x: x[:-1]  # noqa: E731
flat = lambda x: x.flatten(-2)  # noqa: E731
more = lambda x: x[None]  # noqa: E731
none = lambda x: None  # noqa: E731
number = lambda x: 3  # noqa: E731
heads = lambda x: x[..., :1, :]  # noqa: E731
narrow = lambda x: x[..., :D // 2]  # noqa: E731
wide = lambda x: torch.cat([x, x], -1)  # noqa: E731
turned = lambda x: x.transpose(-1, -2).contiguous().transpose(-1, -2)  # noqa: E731
every_other = lambda x: x.repeat_interleave(2)[::2]  # noqa: E731
both = lambda f: dict(kc=f, vc=f)  # noqa: E731
overlapping = lambda x: x[:1].expand(B, -1)  # noqa: E731

FAULTS = {
    "rope": [dict(q=cpu), dict(q=f32), dict(q=half), dict(q=flat), dict(q=more), dict(q=turned), dict(q=none), dict(q=number),
             dict(k=f32), dict(k=short), dict(k=narrow), dict(k=turned), dict(v=none), dict(v=short), dict(v=heads),
             dict(v=f32), dict(pos=none), dict(pos=i64), dict(pos=short), dict(pos=cpu), dict(pos=every_other),
             dict(cos_sin=half), dict(cos_sin=turned), dict(cos_sin=more), dict(wq=f32), dict(wq=short), dict(wk=wide),
             dict(wk=every_other), dict(q_out=short), dict(q_out=f32), dict(k_out=heads), dict(k_out=turned),
             dict(slots=none), dict(slots=i32), dict(slots=short), dict(slots=cpu), both(heads), both(narrow), both(f32),
             dict(kc=short), dict(vc=turned), dict(status=lambda x: torch.zeros(1, dtype=torch.int32)),
             dict(status=lambda x: torch.zeros(1, device="cuda"))],
    "prompt": [dict(q=cpu), dict(q=f32), dict(q=flat), dict(q=turned), dict(k=short), dict(k=narrow), dict(v=heads),
               dict(v=half), dict(v=turned), dict(cu=i64), dict(cu=cpu), dict(cu=more), dict(cu=every_other), dict(out=short),
               dict(out=heads), dict(out=f32), dict(out=turned), dict(out=cpu)],
    "tree": [dict(q=cpu), dict(q=f32), dict(k=short), dict(v=narrow), dict(cu=i64), dict(cu=short), dict(mask=i32),
             dict(mask=short), dict(mask=cpu), dict(mask=every_other), dict(mask=none), both(heads), both(narrow), both(half),
             dict(kc=short), dict(vc=turned), dict(table=i64), dict(table=short), dict(table=flat), dict(table=turned),
             dict(table=overlapping), dict(ctx=i64), dict(ctx=short), dict(ctx=every_other), dict(out=short), dict(out=f32),
             dict(ws=f32), dict(ws=cpu), dict(ws=more)],
    "append": [dict(k=f32), dict(k=cpu), dict(k=none), dict(v=short), dict(v=narrow), dict(v=turned),
               dict(k=short, v=short), dict(k=lambda x: x[0], v=lambda x: x[0]), dict(cu=i64), dict(cu=short), dict(accept=i64),
               dict(accept=short), dict(accept=turned), dict(accept=overlapping), both(heads), both(narrow), both(short),
               both(lambda x: x[0]), dict(table=short), dict(table=i64), dict(ctx=i64), dict(ctx=short), dict(ctx_out=short),
               dict(ctx_out=i64), dict(ctx_out=cpu)],
}


@pytest.mark.parametrize("op,n", [(op, n) for op, faults in FAULTS.items() for n in range(len(faults))],
                         ids=lambda x: str(x))
def test_one_fault_is_refused(op, n):
    error, untouched = call(op, FAULTS[op][n])
    assert error is not None and untouched

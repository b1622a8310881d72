"""Long contexts over the paged cache, as cases to measure.

  attn_shared  attention of drafted trees (one node a sequence: plain decoding) whose sequences share a long prefix by groups
  kv_index     8-bit bounds of the keys of each full page, every layer at once
  attn_select  the pages whose bounds promise the largest scores, for each node and kv head
  attn_sparse  attention of drafted trees over the selected pages

64 query heads of 128 are the layer that o_proj (7168 x 8192) follows; 8 requests of 1 verified + 7 drafted tokens,
1024-token prompts and 5 layers are the serving workload of the bench.  The other sizes are generic.
"""
import math

import torch

own = False  # False: plain torch; True: the library's kernels


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(x) for x in values)


def listed():
    shared = dict(op="attn_shared", hq=64, hkv=8, d=128, page=64)
    index = dict(op="kv_index", hkv=8, d=128, page=64, layers=5)
    select = dict(op="attn_select", hq=64, hkv=8, d=128, page=64, first=1, last=2)
    sparse = dict(op="attn_sparse", hq=64, hkv=8, d=128, page=64)
    return [
        # the draft's verify step: 8 requests behind one system prompt, 8 nodes each: latency
        dict(shared, name="shared_step", groups="8", prefix="1024", tail="64,100,185,287,376,453,476,511",
             nodes="8,8,8,8,8,8,8,8"),
        # small model: three groups of uneven size, two requests of no group, uneven trees
        dict(shared, name="shared_ragged_d64", groups="3,1,5", prefix="640,128,2176", tail="0,5,300,17,1,64,900,33,2,0,777",
             nodes="1,20,3,64,1,8,8,2,31,5,1", hq=12, hkv=4, d=64, page=128),
        # a large decode batch behind a long document: bandwidth and tensor cores
        dict(shared, name="shared_long", groups="64", prefix="16384", tail=_text(100 + 37 * i % 509 for i in range(64)),
             nodes=_text([1] * 64)),
        # after a step's append: the few pages that became full: latency
        dict(index, name="index_step", old="1020,1100,1209,1340,1400,1477,1500,1535", new="1025,1104,1217,1345,1402,1478,1508,1540"),
        # small model, ragged prompts, pages of 16
        dict(index, name="index_ragged_d64", hkv=2, d=64, page=16, layers=3, old="0,0,37,0,512,0", new="1,317,45,1200,512,99"),
        # long documents, just read: bandwidth
        dict(index, name="index_long", old="0,0,0,0", new="16384,16384,16384,16384"),
        # one request, one token, a long document in small pages: latency
        dict(select, name="select_single", ctx="32768", nodes="1", page=16, n_sel=64),
        # the draft's verify step over long contexts
        dict(select, name="select_step", ctx="8192,9001,10240,11111,12345,13579,14000,16383", nodes="8,8,8,8,8,8,8,8", n_sel=16),
        # a large decode batch: bandwidth
        dict(select, name="select_batch", ctx=_text(32768 - 41 * i for i in range(64)), nodes=_text([1] * 64), page=32, n_sel=64),
        # the verify step's attention over the pages it selected
        dict(sparse, name="sparse_step", ctx="8192,9001,10240,11111,12345,13579,14000,16383", nodes="8,8,8,8,8,8,8,8", n_sel=16),
        # small model, uneven trees and contexts, one empty, one shorter than what may be selected
        dict(sparse, name="sparse_ragged_d64", ctx="0,5,777,4095,2048,130", nodes="1,7,3,20,64,1", n_sel=10, hq=14, hkv=2, d=64,
             page=32),
        # a large decode batch: bandwidth
        dict(sparse, name="sparse_batch", ctx=_text(32768 - 997 * i for i in range(32)), nodes=_text([1] * 32), n_sel=32),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    op = rng.choice(["attn_shared", "kv_index", "attn_select", "attn_sparse"])
    c = dict(op=op, hkv=hkv, d=d, page=page)
    if op == "kv_index":
        new = [log(1, 4096) for _ in range(log(1, 16))]
        return dict(c, layers=log(1, 5), old=_text(rng.choice([0, n, max(n - log(1, 64), 0)]) for n in new), new=_text(new))
    c["hq"] = hkv * group
    if op == "attn_shared":
        groups = [log(1, 16) for _ in range(rng.randint(1, 3))]
        b = sum(groups) + rng.randint(0, 2)
        c.update(groups=_text(groups), prefix=_text(log(1, 8192 // page) * page for _ in groups),
                 tail=_text(log(1, 1024) - 1 for _ in range(b)))
    else:
        b = log(1, 16)
        c.update(ctx=_text(log(1, 16384) - 1 for _ in range(b)), n_sel=log(4, 32))
    if op == "attn_select":
        c.update(first=rng.randint(0, 1), last=rng.randint(1, 3))
    nodes, most = [log(1, 32) for _ in range(b)], dict(attn_shared=3e10, attn_select=1e9, attn_sparse=2e9)[op]
    c["nodes"] = _text(nodes)
    while work(c)["flops"] > most and max(nodes) > 1:  # no dearer than the listed ones
        nodes = [(m + 1) // 2 for m in nodes]
        c["nodes"] = _text(nodes)
    return c


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _offsets(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, need):
    """Distinct pages in random order, -1 past a sequence's last one; three pages are nobody's."""
    total = sum(need)
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32).cpu()
    table, at = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total + 3


def _trees(g, nodes):
    """Mask words: node i's parent is one of the nodes before it."""
    r = torch.rand(len(nodes), 64, generator=g, device="cuda").cpu()
    words = []
    for b, m in enumerate(nodes):
        row = [1]
        for i in range(1, m):
            row.append(row[int(r[b, i] * i)] | 1 << i)
        words += row
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op, d, hkv, page = case["op"], case["d"], case["hkv"], case["page"]
    if op == "kv_index":
        old, new, layers = _ints(case["old"]), _ints(case["new"]), case["layers"]
        table, pages = _table(g, [-(-n // page) for n in new])
        s["table"], s["old"], s["new"] = table.cuda(), _int32(old), _int32(new)
        s["kc"] = _randn(g, layers, pages, page, hkv, d)
        s["kc"][..., 3::37] *= 8  # a few large channels, as keys have
        s["vc"] = s["kc"]  # (values are not read)
        s["codes"] = torch.randint(-99, 99, (layers, pages, hkv, 2, d), generator=g, device="cuda", dtype=torch.int8)
        s["exps"] = torch.randint(99, 140, (layers, pages, hkv), generator=g, device="cuda", dtype=torch.uint8)
        full = [int(table[b, j]) for b, (a, n) in enumerate(zip(old, new)) for j in range(a // page, n // page)]
        s["full"] = torch.tensor(full, dtype=torch.long, device="cuda")
    else:
        nodes, hq = _ints(case["nodes"]), case["hq"]
        n = sum(nodes)
        s["cu"], s["max_nodes"] = _offsets(nodes), max(nodes)
        s["q"] = _randn(g, n, hq, d, scale=1.5)
    if op == "attn_shared":
        sizes, prefix, tail = _ints(case["groups"]), _ints(case["prefix"]), _ints(case["tail"])
        of = [i for i, m in enumerate(sizes) for _ in range(m)] + [-1] * (len(tail) - sum(sizes))
        rows, pages = _table(g, [p // page for p in prefix] + [-(-t // page) for t in tail])
        ctx = [t + (prefix[i] if i >= 0 else 0) for i, t in zip(of, tail)]
        table = torch.full((len(tail), max(-(-max(ctx) // page), 1)), -1, dtype=torch.int32)
        for b, i in enumerate(of):
            shared = prefix[i] // page if i >= 0 else 0
            if shared:
                table[b, :shared] = rows[i, :shared]
            m = -(-tail[b] // page)
            table[b, shared:shared + m] = rows[len(prefix) + b, :m]
        s["table"], s["ctx"], s["max_ctx"] = table.cuda(), _int32(ctx), max(ctx)
        s["cu_groups"], s["prefix"] = _offsets(sizes), _int32(prefix)
    elif op != "kv_index":
        ctx = _ints(case["ctx"])
        table, pages = _table(g, [-(-c // page) for c in ctx])
        s["table"], s["ctx"], s["max_ctx"] = table.cuda(), _int32(ctx), max(ctx)
    if op == "attn_select":
        # bounds around a centre a page, with a few wide channels; powers of two as keys of one layer have them
        mid = torch.randn(pages, hkv, 1, d, generator=g, device="cuda") * 22
        wide = (45 + 9 * torch.randn(pages, hkv, 2, d, generator=g, device="cuda")).abs()
        sign = torch.tensor([1.0, -1.0], device="cuda")[:, None]
        s["codes"] = (mid + sign * wide).round().clamp(-127, 127).to(torch.int8)
        s["exps"] = torch.randint(120, 122, (pages, hkv), generator=g, device="cuda", dtype=torch.uint8)
        s["out"] = torch.empty(n, hkv, case["n_sel"], dtype=torch.int32, device="cuda")
    if op in ("attn_shared", "attn_sparse"):
        s["kc"], s["vc"] = _randn(g, pages, page, hkv, d), _randn(g, pages, page, hkv, d)
        s["k"], s["v"] = _randn(g, n, hkv, d), _randn(g, n, hkv, d)
        s["mask"] = _trees(g, nodes)
        s["out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    if op == "attn_sparse":
        # pages as a score of what a sequence's nodes have in common and of their own would select them; the last one always
        n_sel, most = case["n_sel"], s["table"].shape[1]
        seq = torch.repeat_interleave(torch.arange(len(nodes), device="cuda"), torch.tensor(nodes, device="cuda"))
        score = torch.randn(len(nodes), hkv, most, generator=g, device="cuda")[seq]
        score = score + 0.4 * torch.randn(n, hkv, most, generator=g, device="cuda")
        have = (s["ctx"] + page - 1) // page
        j = torch.arange(most, device="cuda")
        score.masked_fill_(j >= have[seq][:, None, None], -math.inf)
        score.masked_fill_(j == (have[seq] - 1)[:, None, None], math.inf)
        best = score.topk(min(n_sel, most), -1)
        sel = best.indices.masked_fill(best.values == -math.inf, 1 << 30).sort(-1).values
        s["sel"] = torch.full((n, hkv, n_sel), -1, dtype=torch.int32, device="cuda")
        s["sel"][..., :sel.shape[2]] = sel.masked_fill(sel == 1 << 30, -1).to(torch.int32)
    s["kv"] = s["index"] = None
    if own:
        import fp8_block_scaled_dynamic_gb300 as mx
        if "kc" in s:
            s["kv"] = mx.KVCache(s["kc"], s["vc"])
        if "codes" in s:
            s["index"] = mx.PageIndex(s["codes"], s["exps"], page)
    return s


def _softmax_plain(sc):
    """In place over the last dim; a row of -inf alone gives zeros."""
    m = sc.amax(-1, keepdim=True)
    sc.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    return sc.div_(sc.sum(-1, keepdim=True).clamp_min(1e-30))


def _pad(cu, most, total):
    """(row index (sequences, most), whether the row is one of the sequence's, and of each packed row its sequence and place)"""
    cu = cu.long()
    i = torch.arange(most, device="cuda")
    idx, real = cu[:-1, None] + i, i < (cu[1:] - cu[:-1])[:, None]
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, at, right=True) - 1
    return idx.clamp_max(total - 1), real, seq, at - cu[seq]


def _exponent(amax):
    """The least whole e >= -100 with amax <= 127 * 2^e."""
    _, e = torch.frexp(amax)  # amax = f 2^e, 1/2 <= f < 1
    e = torch.where(amax == 0, -100, e - 7)
    e = torch.where(torch.ldexp(amax, -e) > 127, e + 1, e)
    return e.clamp_min(-100)


def _plain(s):
    op, d, hkv, page = s["op"], s["d"], s["hkv"], s["page"]
    if op == "kv_index":
        x = s["kc"][:, s["full"]].float()  # (layers, full pages, page, hkv, d)
        e = _exponent(x.abs().amax((2, 4)))[..., None]
        s["codes"][:, s["full"], :, 0] = torch.ldexp(x.amax(2), -e).ceil().to(torch.int8)
        s["codes"][:, s["full"], :, 1] = torch.ldexp(x.amin(2), -e).floor().to(torch.int8)
        s["exps"][:, s["full"]] = (e[..., 0] + 127).to(torch.uint8)
        return s["codes"], s["exps"]
    t, hq = s["q"].shape[0], s["hq"]
    idx, real, seq, at = _pad(s["cu"], s["max_nodes"], t)
    n, m = idx.shape
    tab = s["table"][:, :max(-(-s["max_ctx"] // page), 1)].long().clamp_min(0)
    if op == "attn_select":
        q = s["q"].float().view(t, hkv, -1, d)
        q = torch.ldexp(q, -_exponent(q.abs().amax((2, 3)))[..., None, None]).round()
        # whole numbers below 2^24: the sums are exact
        q = torch.cat([q.clamp_min(0), q.clamp_max(0)], -1)[idx]  # (n, m, hkv, group, 2d)
        b = s["codes"][tab].flatten(-2).float()  # (n, pages, hkv, 2d)
        q = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, 2 * d)
        sc = torch.matmul(q, b.permute(0, 2, 3, 1)).view(n, hkv, m, -1, b.shape[1]).amax(3)
        sc = torch.ldexp(sc, s["exps"][tab].permute(0, 2, 1)[:, :, None].int() - 127)
        have = ((s["ctx"] + page - 1) // page)[:, None, None, None]
        j = torch.arange(b.shape[1], device="cuda")
        sc = sc.masked_fill((j < s["first"]) | (j >= have - s["last"]), math.inf).masked_fill(j >= have, -math.inf)
        best = torch.sort(sc, dim=-1, descending=True, stable=True)  # (of equal ones, the lowest page first)
        k = min(s["n_sel"], b.shape[1])
        pick = best.indices[..., :k].masked_fill(best.values[..., :k] == -math.inf, 1 << 30).sort(-1).values
        out = torch.full((n, hkv, m, s["n_sel"]), -1, dtype=torch.int32, device="cuda")
        out[..., :k] = pick.masked_fill(pick == 1 << 30, -1).to(torch.int32)
        return out[seq, :, at]
    new = (s["mask"][idx][:, :, None] >> torch.arange(m, device="cuda") & 1).bool() & real[:, None]
    if op == "attn_shared":
        q = s["q"][idx].float().view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
        cols = tab.shape[1]
        keys = torch.cat([s["kc"][tab].view(n, cols * page, hkv, d), s["k"][idx]], 1).float()
        vals = torch.cat([s["vc"][tab].view(n, cols * page, hkv, d), s["v"][idx]], 1).float()
        sc = torch.matmul(q, keys.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
        old = torch.arange(cols * page, device="cuda") < s["ctx"][:, None]
        see = torch.cat([old[:, None].expand(-1, m, -1), new], 2)
        sc.view(n, hkv, -1, *see.shape[1:]).masked_fill_(~see[:, None, None], float("-inf"))
        o = torch.matmul(_softmax_plain(sc), vals.permute(0, 2, 1, 3))
        return o.view(n, hkv, -1, m, d).permute(0, 3, 1, 2, 4).reshape(n, m, hq, d)[seq, at].to(torch.bfloat16)
    sel = s["sel"].long()  # (t, hkv, n_sel)
    head = torch.arange(hkv, device="cuda")[:, None]
    pg = tab[seq[:, None, None], sel.clamp(0, tab.shape[1] - 1)]
    tok = sel[..., None] * page + torch.arange(page, device="cuda")
    old = ((sel >= 0)[..., None] & (tok < s["ctx"][seq][:, None, None, None])).flatten(-2)
    see = torch.cat([old, new[seq, at][:, None].expand(-1, hkv, -1)], -1)

    def rows(cache, x):
        c = cache.transpose(1, 2)[pg, head].reshape(t, hkv, -1, d)
        return torch.cat([c, x[idx][seq].transpose(1, 2)], 2).float()

    q = s["q"].float().view(t, hkv, -1, d)
    sc = torch.matmul(q, rows(s["kc"], s["k"]).transpose(2, 3)).mul_(1 / math.sqrt(d))
    sc.masked_fill_(~see[:, :, None], float("-inf"))
    return torch.matmul(_softmax_plain(sc), rows(s["vc"], s["v"])).view(t, hq, d).to(torch.bfloat16)


def run(s):
    if not own:
        return _plain(s)
    import fp8_block_scaled_dynamic_gb300 as mx
    op = s["op"]
    if op == "kv_index":
        mx.kv_index(s["kv"], s["index"], s["table"], s["old"], s["new"])
        return s["codes"], s["exps"]
    if op == "attn_select":
        return mx.attn_select(s["q"], s["cu"], s["index"], s["table"], s["ctx"], s["n_sel"], first=s["first"], last=s["last"],
                              out=s["out"])
    if op == "attn_shared":
        return mx.attn_shared(s["q"], s["k"], s["v"], s["cu"], s["mask"], s["kv"], s["table"], s["ctx"], s["cu_groups"],
                              s["prefix"], out=s["out"])
    return mx.attn_sparse(s["q"], s["k"], s["v"], s["cu"], s["mask"], s["kv"], s["table"], s["ctx"], s["sel"], out=s["out"])


def work(case):
    d, hkv, page, op = case["d"], case["hkv"], case["page"], case["op"]
    if op == "kv_index":
        full = sum(n // page - a // page for a, n in zip(_ints(case["old"]), _ints(case["new"])))
        return {"bytes": full * case["layers"] * hkv * (2 * page * d + 2 * d + 1), "flops": 3 * full * case["layers"] * hkv * page * d}
    nodes, hq = _ints(case["nodes"]), case["hq"]
    n = sum(nodes)
    if op == "attn_shared":  # a node sees, of a random tree, about ln(n) nodes: counted as itself alone
        sizes, prefix, tail = _ints(case["groups"]), _ints(case["prefix"]), _ints(case["tail"])
        own_prefix = [p for p, m in zip(prefix, sizes) for _ in range(m)] + [0] * (len(tail) - sum(sizes))
        return {"bytes": 4 * (sum(prefix) + sum(tail) + n) * hkv * d + 4 * n * hq * d,
                "flops": 4 * d * hq * sum(m * (p + t + 1) for p, t, m in zip(own_prefix, tail, nodes))}
    ctx = _ints(case["ctx"])
    have = [-(-c // page) for c in ctx]
    if op == "attn_select":
        return {"bytes": sum(have) * hkv * (2 * d + 1) + 2 * n * hq * d + 4 * n * hkv * case["n_sel"],
                "flops": 2 * d * hq * sum(p * m for p, m in zip(have, nodes))}
    # of each sequence the pages that its first node selects: the others' own ones depend on the inputs
    seen = [min(c, case["n_sel"] * page) for c in ctx]
    return {"bytes": 4 * (sum(seen) + n) * hkv * d + 4 * n * hq * d + 4 * n * hkv * case["n_sel"],
            "flops": 4 * d * hq * sum(m * (c + 1) for c, m in zip(seen, nodes))}


def exact(case, seed):
    """From the definitions, in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    op, d, hkv, page = s["op"], s["d"], s["hkv"], s["page"]

    def power(top):  # by search: no logarithms
        e = torch.full(top.shape, -100.0, dtype=torch.float64, device="cuda")
        for _ in range(240):
            e = e + (top > 127 * torch.pow(2.0, e))
        return e

    if op == "kv_index":
        table = s["table"].tolist()
        for b, (a, n) in enumerate(zip(_ints(case["old"]), _ints(case["new"]))):
            of = table[b][a // page:n // page]
            if not of:
                continue
            x = s["kc"][:, of].double().permute(1, 0, 3, 2, 4)  # (pages, layers, hkv, page, d)
            e = power(x.abs().flatten(-2).max(-1).values)
            scaled = x / torch.pow(2.0, e)[..., None, None]
            s["codes"][:, of, :, 0] = scaled.max(-2).values.ceil().to(torch.int8).transpose(0, 1)
            s["codes"][:, of, :, 1] = scaled.min(-2).values.floor().to(torch.int8).transpose(0, 1)
            s["exps"][:, of] = (e + 127).to(torch.uint8).transpose(0, 1)
        return s["codes"], s["exps"]
    nodes, hq, table = _ints(case["nodes"]), s["hq"], s["table"].long()
    g, ctx, a = hq // hkv, s["ctx"].tolist(), 0
    if op == "attn_select":
        out = torch.full((sum(nodes), hkv, s["n_sel"]), -1, dtype=torch.int32, device="cuda")
        for c, m, row in zip(ctx, nodes, table):
            p = -(-c // page)
            always = [j for j in range(p) if j < s["first"] or j >= p - s["last"]]
            rest = [j for j in range(p) if s["first"] <= j < p - s["last"]]
            for h in range(hkv):
                x = s["q"][a:a + m, h * g:(h + 1) * g].double()
                x = (x / torch.pow(2.0, power(x.abs().amax((1, 2))))[:, None, None]).round()
                hi, lo = (s["codes"][row[:p], h, i].double() for i in (0, 1))
                size = torch.pow(2.0, s["exps"][row[:p], h].double() - 127)
                bound = torch.stack([(torch.where(x[:, i] > 0, x[:, i], 0.0) @ hi.T + torch.where(x[:, i] < 0, x[:, i], 0.0) @ lo.T)
                                     for i in range(g)]).amax(0) * size
                for i, v in enumerate(bound.tolist()):
                    best = sorted(rest, key=lambda j: (-v[j], j))[:max(s["n_sel"] - len(always), 0)]
                    pick = sorted(always + best)
                    out[a + i, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            a += m
        return out
    o, words = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["mask"].tolist()
    for b, (c, m) in enumerate(zip(ctx, nodes)):
        tok = torch.arange(c, device="cuda")
        pg = table[b][tok // page] if c else tok
        new = torch.tensor([[w >> j & 1 for j in range(m)] for w in words[a:a + m]], dtype=torch.bool, device="cuda")
        for h in range(hkv):
            if op == "attn_sparse":
                seen = torch.zeros(m, c // page + 2, dtype=torch.bool, device="cuda")
                pick = s["sel"][a:a + m, h].long()
                seen.scatter_(1, torch.where(pick < 0, c // page + 1, pick), True)
                keep = seen[:, tok // page] if c else torch.zeros(m, 0, dtype=torch.bool, device="cuda")
                some = keep.any(0)
                k, v = (torch.cat([s[x + "c"][pg[some], tok[some] % page, h], s[x][a:a + m, h]]).double() for x in "kv")
                see = torch.cat([keep[:, some], new], 1)
            else:
                k, v = (torch.cat([s[x + "c"][pg, tok % page, h], s[x][a:a + m, h]]).double() for x in "kv")
                see = torch.cat([torch.ones(m, c, dtype=torch.bool, device="cuda"), new], 1)
            q = s["q"][a:a + m, h * g:(h + 1) * g].double()
            p = torch.einsum("mgd,kd->gmk", q, k) / math.sqrt(d)
            p.masked_fill_(~see, -math.inf)
            o[a:a + m, h * g:(h + 1) * g] = (torch.softmax(p, -1) @ v).transpose(0, 1)
        a += m
    return o

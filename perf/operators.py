"""The attention operators between the qkv projection and o_proj, as cases to measure.

  qk_norm_rope  RMS norm of every query and key head, the position rotation, and the write of k and v into cache pages
  attn_prompt   causal attention of packed prompts with grouped heads
  attn_tree     attention of a tree of drafted tokens over a paged cache (one node a sequence: plain decoding)
  kv_append     the accepted nodes' keys and values into the cache, all layers in one call

64 query heads of 128 are the layer that o_proj (7168 x 8192) follows; 8 requests of 1 verified + 7 drafted tokens
and 1024-token prompts are the serving workload of the bench.  The other sizes are generic.
"""
import math

import torch

own = False  # False: plain torch; True: the library's kernels


def _ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    rope = dict(op="qk_norm_rope", hq=64, hkv=8, d=128, rot=128, interleaved=False, cache=False)
    prompt = dict(op="attn_prompt", hq=64, hkv=8, d=128)
    tree = dict(op="attn_tree", hq=64, hkv=8, d=128, page=64)
    app = dict(op="kv_append", hkv=8, d=128, page=64)
    return [
        # one draft step of 8 requests (1 verified + 7 drafted tokens each): latency
        dict(rope, name="rope_step", lens="8,8,8,8,8,8,8,8"),
        # small model, ragged prompts, half of each head rotated, neighbouring pairs, into the cache
        dict(rope, name="rope_ragged_d64", lens="1,317,45,1200,2,99", hq=14, hkv=2, d=64, rot=32, interleaved=True,
             cache=True),
        # 8 prompts of 1024 tokens, into the cache: bandwidth
        dict(rope, name="rope_prompts", lens="1024,1024,1024,1024,1024,1024,1024,1024", cache=True),
        # one 1024-token prompt
        dict(prompt, name="prompt_1k", lens="1024"),
        # a batch of chats of uneven length, one of a single token, smaller heads
        dict(prompt, name="prompt_ragged_d64", lens="1,37,513,2047,130,900", hq=14, hkv=2, d=64),
        # long document: tensor cores
        dict(prompt, name="prompt_8k", lens="8192"),
        # plain decoding of one request: latency
        dict(tree, name="tree_single", ctx="1500", nodes="1"),
        # the draft's verify step: 8 requests, 8 nodes each, around 1024 + 512 tokens in the cache
        dict(tree, name="tree_step", ctx="1024,1100,1209,1311,1400,1477,1500,1535", nodes="8,8,8,8,8,8,8,8"),
        # long contexts with wide trees of uneven size: bandwidth, then tensor cores
        dict(tree, name="tree_long", ctx="32768,30001,0,16385,24576,31999,8191,32000,129,20000",
             nodes="32,17,5,64,32,1,40,32,9,32", page=16),
        # small model, few cached tokens, one request with none, uneven trees
        dict(tree, name="tree_ragged_d64", ctx="0,5,777,4095,1", nodes="1,64,3,20,7", hq=12, hkv=4, d=64, page=128),
        # what the draft accepted, five layers
        dict(app, name="append_step", layers=5, ctx="1024,1100,1209,1311,1400,1477,1500,1535", nodes="8,8,8,8,8,8,8,8",
             most=8),
        # a large batch, 32 layers, pages of 16
        dict(app, name="append_batch", layers=32, ctx=",".join(str(7 + 3 * i % 120) for i in range(64)),
             nodes=",".join(["8"] * 64), most=8, page=16),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    op = rng.choice(["qk_norm_rope", "attn_prompt", "attn_tree", "kv_append"])
    if op == "qk_norm_rope":
        n = log(1, 8)
        return dict(op=op, hq=hkv * group, hkv=hkv, d=d, rot=rng.choice([d, d // 2, 16]), interleaved=rng.random() < 0.5,
                    cache=rng.random() < 0.5, lens=",".join(str(log(1, 1024)) for _ in range(n)))
    if op == "attn_prompt":
        n = log(1, 8)
        return dict(op=op, hq=hkv * group, hkv=hkv, d=d, lens=",".join(str(log(1, 8192 // n)) for _ in range(n)))
    n = log(1, 16)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "attn_tree":
        return dict(op=op, hq=hkv * group, hkv=hkv, d=d, page=page,
                    ctx=",".join(str(log(1, 16384) - 1) for _ in range(n)),
                    nodes=",".join(str(log(1, 64)) for _ in range(n)))
    return dict(op=op, hkv=hkv, d=d, page=page, layers=log(1, 32), most=rng.randint(1, 9),
                ctx=",".join(str(log(1, 1024) - 1) for _ in range(n)),
                nodes=",".join(str(log(1, 64)) for _ in range(n)))


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _offsets(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def _pages(g, need, page):
    """A table (sequences, most pages) of distinct pages in random order, -1 past a sequence's last one."""
    most, total = max(need), sum(need)
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32).cpu()
    table, at = torch.full((len(need), max(most, 1)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), total + 3


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "qk_norm_rope":
        lens = _ints(case["lens"])
        t, hq, rot = sum(lens), case["hq"], case["rot"]
        # the packed output of the qkv projection, with a few large channels as activations have
        qkv = _randn(g, t, hq + 2 * hkv, d)
        qkv[:, :, 3::37] *= 8
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["wq"], s["wk"] = (1 + 0.2 * _randn(g, d).float()).bfloat16(), (1 + 0.2 * _randn(g, d).float()).bfloat16()
        start = torch.randint(0, 2048, (len(lens),), generator=g, device="cuda")
        off = _offsets(lens).long()
        seq = torch.searchsorted(off, torch.arange(t, device="cuda"), right=True) - 1
        pos = start[seq] + torch.arange(t, device="cuda") - off[seq]
        s["pos"] = pos.to(torch.int32)
        p = torch.arange(2048 + max(lens), device="cuda", dtype=torch.float64)
        ang = p[:, None] * (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot))
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"].contiguous()), torch.empty_like(s["k"].contiguous())
        s["kc"] = s["vc"] = s["slots"] = s["kv"] = None
        if case["cache"]:
            pages = (t + 63) // 64 + 2
            s["kc"], s["vc"] = _randn(g, pages, 64, hkv, d), _randn(g, pages, 64, hkv, d)
            s["slots"] = torch.randperm(pages * 64, generator=g, device="cuda")[:t]
        s["eps"] = 1e-6
    elif case["op"] == "attn_prompt":
        lens = _ints(case["lens"])
        t, hq = sum(lens), case["hq"]
        s["q"], s["k"] = _randn(g, t, hq, d, scale=1.5), _randn(g, t, hkv, d)
        s["v"] = _randn(g, t, hkv, d)
        s["cu"], s["max_len"] = _offsets(lens), max(lens)
        s["out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
    else:
        ctx, nodes = _ints(case["ctx"]), _ints(case["nodes"])
        n, page = sum(nodes), case["page"]
        room = [c + (case.get("most", 0)) for c in ctx]
        s["table"], pages = _pages(g, [-(-r // page) for r in room], page)
        s["ctx"], s["cu"] = torch.tensor(ctx, dtype=torch.int32, device="cuda"), _offsets(nodes)
        if case["op"] == "attn_tree":
            hq = case["hq"]
            s["kc"], s["vc"] = _randn(g, pages, page, hkv, d), _randn(g, pages, page, hkv, d)
            s["q"] = _randn(g, n, hq, d, scale=1.5)
            s["k"], s["v"] = _randn(g, n, hkv, d), _randn(g, n, hkv, d)
            r = torch.rand(len(nodes), 64, generator=g, device="cuda").cpu()
            words = []
            for b, m in enumerate(nodes):  # node i's parent is one of the nodes before it
                row = [1]
                for i in range(1, m):
                    row.append(row[int(r[b, i] * i)] | 1 << i)
                words += row
            s["mask"] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")
            s["out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
            s["max_ctx"], s["max_nodes"] = max(ctx), max(nodes)
        else:
            layers, most = case["layers"], case["most"]
            s["kc"], s["vc"] = _randn(g, layers, pages, page, hkv, d), _randn(g, layers, pages, page, hkv, d)
            s["k"], s["v"] = _randn(g, layers, n, hkv, d), _randn(g, layers, n, hkv, d)
            r = torch.rand(len(nodes), 65, generator=g, device="cuda").cpu()
            acc = torch.full((len(nodes), most), -1, dtype=torch.int32)
            for b, m in enumerate(nodes):  # a rising path through the tree
                path = [i for i in range(m) if i == 0 or r[b, i] < 0.6][:most]
                acc[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
            s["accept"] = acc.cuda()
            s["ctx_out"] = torch.empty_like(s["ctx"])
    if own and s.get("kc") is not None:
        import fp8_block_scaled_dynamic_gb300 as mx
        s["kv"] = mx.KVCache(s["kc"], s["vc"])
    return s


def _rope_plain(x, w, s):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    rot = s["rot"]
    cs = s["cos_sin"][s["pos"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


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


def _plain(s):
    op, d, hkv = s["op"], s["d"], s["hkv"]
    if op == "qk_norm_rope":
        q, k = _rope_plain(s["q"], s["wq"], s), _rope_plain(s["k"], s["wk"], s)
        if s["cache"]:
            s["kc"].view(-1, hkv, d)[s["slots"]] = k
            s["vc"].view(-1, hkv, d)[s["slots"]] = s["v"]
            return q, k, s["kc"], s["vc"]
        return q, k
    if op == "attn_prompt":
        t, hq = s["q"].shape[0], s["hq"]
        idx, real, seq, at = _pad(s["cu"], s["max_len"], t)
        n, l = idx.shape
        q = s["q"][idx].float().view(n, l, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
        sc = torch.matmul(q, s["k"][idx].float().permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
        i = torch.arange(l, device="cuda")
        sc.view(n, hkv, -1, l, l).masked_fill_(i > i[:, None], float("-inf"))
        o = torch.matmul(_softmax_plain(sc), s["v"][idx].float().permute(0, 2, 1, 3))
        return o.view(n, hkv, -1, l, d).permute(0, 3, 1, 2, 4).reshape(n, l, hq, d)[seq, at].to(torch.bfloat16)
    if op == "attn_tree":
        t, hq, page = s["q"].shape[0], s["hq"], s["page"]
        idx, real, seq, at = _pad(s["cu"], s["max_nodes"], t)
        n, m = idx.shape
        q = s["q"][idx].float().view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
        cols = -(-s["max_ctx"] // page)
        tab = s["table"][:, :cols].long().clamp_min(0)
        keys = torch.cat([s["kc"][tab].view(n, cols * page, hkv, d), s["k"][idx]], 1).float()
        vals = torch.cat([s["vc"][tab].view(n, cols * page, hkv, d), s["v"][idx]], 1).float()
        sc = torch.matmul(q, keys.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
        old = torch.arange(cols * page, device="cuda") < s["ctx"][:, None]
        new = (s["mask"][idx][:, :, None] >> torch.arange(m, device="cuda") & 1).bool() & real[:, None]
        see = torch.cat([old[:, None].expand(-1, m, -1), new], 2)
        sc.view(n, hkv, -1, *see.shape[1:]).masked_fill_(~see[:, None, None], float("-inf"))
        o = torch.matmul(_softmax_plain(sc), vals.permute(0, 2, 1, 3))
        return o.view(n, hkv, -1, m, d).permute(0, 3, 1, 2, 4).reshape(n, m, hq, d)[seq, at].to(torch.bfloat16)
    page, acc = s["page"], s["accept"].long()
    ok = acc >= 0
    at = s["ctx"].long()[:, None] + torch.arange(acc.shape[1], device="cuda")
    b, i = ok.nonzero(as_tuple=True)
    src, at = s["cu"].long()[b] + acc[b, i], at[b, i]
    pg, sl = s["table"][b, at // page].long(), at % page
    s["kc"][:, pg, sl] = s["k"][:, src]
    s["vc"][:, pg, sl] = s["v"][:, src]
    return s["kc"], s["vc"], s["ctx"] + ok.sum(1).to(torch.int32)


def run(s):
    if not own:
        return _plain(s)
    import fp8_block_scaled_dynamic_gb300 as mx
    op = s["op"]
    if op == "qk_norm_rope":
        q, k = mx.qk_norm_rope(s["q"], s["k"], s["pos"], s["cos_sin"], wq=s["wq"], wk=s["wk"], eps=s["eps"],
                               interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"],
                               v=s["v"] if s["kv"] else None, cache=s["kv"], slots=s["slots"])
        return (q, k, s["kc"], s["vc"]) if s["kv"] else (q, k)
    if op == "attn_prompt":
        return mx.attn_prompt(s["q"], s["k"], s["v"], s["cu"], out=s["out"])
    if op == "attn_tree":
        return mx.attn_tree(s["q"], s["k"], s["v"], s["cu"], s["mask"], s["kv"], s["table"], s["ctx"], out=s["out"])
    ctx = mx.kv_append(s["k"], s["v"], s["cu"], s["accept"], s["kv"], s["table"], s["ctx"], ctx_out=s["ctx_out"])
    return s["kc"], s["vc"], ctx


def work(case):
    d, hkv, op = case["d"], case["hkv"], case["op"]
    if op == "qk_norm_rope":
        lens = _ints(case["lens"])
        t, heads = sum(lens), case["hq"] + hkv
        moved = 2 * t * heads * d + (3 * t * hkv * d if case["cache"] else 0)  # values; the cache: v read, k and v written
        return {"bytes": 2 * moved + 4 * case["rot"] * max(lens), "flops": t * heads * (4 * d + 3 * case["rot"])}
    if op == "attn_prompt":
        lens, hq = _ints(case["lens"]), case["hq"]
        return {"bytes": 4 * sum(lens) * (hq + hkv) * d, "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    ctx, nodes = _ints(case["ctx"]), _ints(case["nodes"])
    if op == "attn_tree":  # a node sees the context and, of a random tree, about ln(n) nodes: counted as itself alone
        hq = case["hq"]
        return {"bytes": 4 * (sum(ctx) + sum(nodes)) * hkv * d + 4 * sum(nodes) * hq * d,
                "flops": 4 * d * hq * sum(n * (c + 1) for c, n in zip(ctx, nodes))}
    rows = sum(min(case["most"], 1 + 0.6 * (n - 1)) for n in nodes)  # of the nodes, 0.6 are accepted
    return {"bytes": 8 * rows * hkv * d * case["layers"], "flops": 0}


def exact(case, seed):
    """From the definitions, in 64 bits, head by head and sequence by sequence."""
    s = prepare(case, seed)
    op, d, hkv = s["op"], s["d"], s["hkv"]
    if op == "qk_norm_rope":
        cs, rot = s["cos_sin"].double()[s["pos"].long()], s["rot"]
        half = rot // 2

        def rope(x, w):
            x = x.double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * w.double()
            y = x.clone()
            for j in range(half):
                a, b = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + half)
                c, n = cs[:, j, None], cs[:, half + j, None]
                y[..., a], y[..., b] = x[..., a] * c - x[..., b] * n, x[..., a] * n + x[..., b] * c
            return y

        q, k = rope(s["q"], s["wq"]), rope(s["k"], s["wk"])
        if not s["cache"]:
            return q, k
        kc, vc = s["kc"].double(), s["vc"].double()
        kc.view(-1, hkv, d)[s["slots"]], vc.view(-1, hkv, d)[s["slots"]] = k, s["v"].double()
        return q, k, kc, vc
    if op == "attn_prompt":
        o, lens, hq = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), _ints(s["lens"]), s["hq"]
        a = 0
        for n in lens:
            low = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
            for h in range(hq):
                k, v = (s[x][a:a + n, h // (hq // hkv)].double() for x in "kv")
                p = (s["q"][a:a + n, h].double() @ k.T / math.sqrt(d)).where(low, torch.tensor(-math.inf, device="cuda", dtype=torch.float64))
                o[a:a + n, h] = torch.softmax(p, -1) @ v
            a += n
        return o
    ctx, nodes, page = _ints(case["ctx"]), _ints(case["nodes"]), s["page"]
    if op == "attn_tree":
        hq = s["hq"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        words, a = s["mask"].tolist(), 0
        for b, (c, m) in enumerate(zip(ctx, nodes)):
            at = torch.arange(c, device="cuda")
            pg = s["table"][b].long()[at // page] if c else at
            see = torch.tensor([[w >> j & 1 for j in range(m)] for w in words[a:a + m]], dtype=torch.bool, device="cuda")
            see = torch.cat([torch.ones(m, c, dtype=torch.bool, device="cuda"), see], 1)
            for h in range(hkv):
                k, v = (torch.cat([s[x + "c"][pg, at % page, h], s[x][a:a + m, h]]).double() for x in "kv")
                q = s["q"][a:a + m, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
                p = torch.einsum("mgd,kd->gmk", q, k) / math.sqrt(d)
                p.masked_fill_(~see, -math.inf)
                o[a:a + m, h * (hq // hkv):(h + 1) * (hq // hkv)] = (torch.softmax(p, -1) @ v).transpose(0, 1)
            a += m
        return o
    kc, vc, table, acc, a = s["kc"].double(), s["vc"].double(), s["table"].tolist(), s["accept"].tolist(), 0
    for b, (c, m) in enumerate(zip(ctx, nodes)):
        for i, j in enumerate(x for x in acc[b] if x >= 0):
            kc[:, table[b][(c + i) // page], (c + i) % page] = s["k"][:, a + j].double()
            vc[:, table[b][(c + i) // page], (c + i) % page] = s["v"][:, a + j].double()
        a += m
    return kc, vc, None

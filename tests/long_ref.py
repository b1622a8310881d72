"""The long-context operators from their definitions: attention in 64 bits
(with attn_ref's bounds), bounds and choices of pages in whole numbers."""
import math

import torch

import attn_ref


def shared_table(table, groups, prefix, page):
    """The block table with every sequence's prefix read from its group's first row."""
    t, b = table.clone(), 0
    for n, p in zip(groups, prefix):
        cols = p // page
        t[b:b + n, :cols] = table[b, :cols]
        b += n
    return t


def seen_rows(q, keys, vals, scale):
    """attn_ref.rows where every key is seen; an infinity in v stays one (the
    weights are positive), unless it meets the other one or a NaN."""
    o, bound = attn_ref.rows(q, keys, vals, torch.ones(q.shape[0], keys.shape[0], dtype=torch.bool, device=q.device), scale)
    if bool(torch.isfinite(vals).all()):
        return o, bound
    nan, up, down = torch.isnan(vals).any(0), (vals == math.inf).any(0), (vals == -math.inf).any(0)
    for mask, x in [(up & ~down & ~nan, math.inf), (down & ~up & ~nan, -math.inf)]:
        o = torch.where(mask & ~torch.isnan(bound), torch.full_like(o, x), o)
    return o, bound


def assert_within(got, want, bound, what):
    """attn_ref's, with infinities where the definition has them."""
    inf = torch.isinf(want)
    assert bool((got.double()[inf] == want[inf]).all()), f"{what}: infinities"
    attn_ref.assert_within(got.masked_fill(inf, 0.0), want.masked_fill(inf, 0.0), bound, what)


def sparse(q, k, v, nodes, mask, kc, vc, table, ctx, sel, scale):
    """attn_sparse: yields (rows, o, bound) a sequence."""
    G, a, page, Hkv = q.shape[1] // k.shape[1], 0, kc.shape[1], k.shape[1]
    dev = q.device
    for b, (n, c) in enumerate(zip(nodes, ctx)):
        if n:
            have = -(-c // page)
            words = mask[a:a + n].tolist()
            new = torch.tensor([[w >> i & 1 for i in range(n)] for w in words], dtype=torch.bool, device=dev)
            os, bs = [], []
            for h in range(Hkv):
                pick = sel[a:a + n, h].long()
                seen = torch.zeros(n, have + 1, dtype=torch.bool, device=dev)
                seen.scatter_(1, torch.where((pick < 0) | (pick >= have), have, pick), True)
                seen[:, have] = False
                some = seen.any(0).nonzero()[:, 0]  # logical pages
                j = (some[:, None] * page + torch.arange(page, device=dev)).flatten()
                j = j[j < c]
                pg = table[b].long()[j // page]
                ok = (pg >= 0) & (pg < kc.shape[0])
                pg = torch.where(ok, pg, torch.zeros_like(pg))
                see = torch.cat([seen[:, j // page], new], 1)
                ks = torch.cat([torch.where(ok[:, None], kc[pg, j % page, h], 0), k[a:a + n, h]]).double()
                vs = torch.cat([torch.where(ok[:, None], vc[pg, j % page, h], 0), v[a:a + n, h]]).double()
                for g in range(G):
                    # (a key that a row does not see has no part in it, whatever it holds: row by row)
                    ob = [seen_rows(q[a + i:a + i + 1, h * G + g].double(), ks[see[i]], vs[see[i]], scale) for i in range(n)]
                    os.append(torch.cat([x[0] for x in ob]))
                    bs.append(torch.cat([x[1] for x in ob]))
            yield torch.arange(a, a + n, device=dev), torch.stack(os, 1), torch.stack(bs, 1)
        a += n


def exponent(amax):
    """The least whole e >= -100 with amax <= 127 * 2^e."""
    e = -100
    while amax > 127 * 2.0 ** e:
        e += 1
    return e


def bounds(keys):
    """(codes (2, D), code) of a page's keys (tokens, D) of one head."""
    x = keys.double().cpu()
    if not bool(torch.isfinite(x).all()):
        return torch.zeros(2, x.shape[1], dtype=torch.int8), 255
    e = exponent(float(x.abs().max()))
    up, down = (x.max(0).values / 2.0 ** e).ceil(), (x.min(0).values / 2.0 ** e).floor()
    return torch.stack([up, down]).to(torch.int8), e + 127


def whole(q):
    """A group's q (G, D) in whole numbers."""
    x = q.double().cpu()
    if not bool(torch.isfinite(x).all()):
        return torch.zeros(x.shape, dtype=torch.int64)
    return (x / 2.0 ** exponent(float(x.abs().max()))).round().long()  # (ties to even)


def select(q, nodes, codes, exps, table, ctx, page, n_sel, first, last, N):
    """(N, Hkv, n_sel); rows past the last sequence are -7."""
    Hkv = codes.shape[1]
    G = q.shape[1] // Hkv
    out = torch.full((N, Hkv, n_sel), -7, dtype=torch.int32)
    codes, exps, table, a = codes.cpu().long(), exps.cpu().tolist(), table.cpu().tolist(), 0
    for b, (n, c) in enumerate(zip(nodes, ctx)):
        P = -(-c // page)
        for i in range(a, a + n):
            for h in range(Hkv):
                x = whole(q[i, h * G:(h + 1) * G])
                always = [j for j in range(P) if j < first or j >= P - last]
                rest = []
                for j in range(P):
                    if first <= j < P - last:
                        pg = table[b][j]
                        if not 0 <= pg < codes.shape[0]:
                            s = 0.0
                        elif exps[pg][h] == 255:
                            s = math.inf
                        else:
                            up, down = codes[pg, h]
                            s = int((x.clamp_min(0) * up + x.clamp_max(0) * down).sum(1).max()) * 2.0 ** (exps[pg][h] - 127)
                        rest.append((-s, j))
                pick = sorted(always + [j for _, j in sorted(rest)[:max(n_sel - len(always), 0)]]) if P > n_sel else list(range(P))
                out[i, h] = torch.tensor(pick + [-1] * (n_sel - len(pick)), dtype=torch.int32)
        a += n
    return out

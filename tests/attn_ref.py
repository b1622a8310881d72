"""Attention, norm and rotation in 64 bits, written from the definitions, with
the error bounds the tests hold the kernels to."""
import math

import torch

BF16 = 2.0 ** -8   # the relative error of one rounding to bf16 (8 bits)


def rows(q, keys, vals, see, scale):
    """Softmax rows: q (M, D), keys/vals (K, D) float64, see (M, K) bool.
    Returns (o, bound): a row that sees nothing is 0; what is not seen has no
    part in the row, NaN included.

    The bound of one element, from the kernels' arithmetic: o is rounded to
    bf16 (2^-8 |o|); every softmax weight is rounded to bf16 before its product
    with v, not in their fp32 sum (2^-8 sum p|v|); the scores are fp32 sums of D
    products (relative to sum |q||k|: D 2^-23), and an error delta of a score
    moves its weight by 2 delta; the exponential and the running rescales stay
    within 2^-18."""
    M, D = q.shape
    s = (q @ keys.T) * scale
    mag = ((q.abs() @ keys.abs().T) * abs(scale)).masked_fill(~see, 0.0)
    s = s.masked_fill(~see, -math.inf)
    m = s.amax(1, keepdim=True) if s.shape[1] else torch.full((M, 1), -math.inf, dtype=s.dtype, device=s.device)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(1, keepdim=True)
    p = torch.where(l > 0, p / l.clamp_min(1e-300), p)
    clean = torch.nan_to_num(vals, nan=0.0, posinf=0.0, neginf=0.0)
    o = p @ clean
    # a row is NaN where it sees a NaN or an infinity
    poison = see.double() @ (~torch.isfinite(vals)).double()
    delta = D * 2.0 ** -23 * mag.amax(1, keepdim=True) if mag.shape[1] else 0.0
    bound = BF16 * o.abs() + (BF16 + 4 * delta + 2.0 ** -18) * (p @ clean.abs()) + 1e-30
    return torch.where(poison > 0, torch.full_like(o, math.nan), o), bound


def prompt(q, k, v, lens, scale, rows_of=None):
    """Causal attention of packed sequences; rows_of: of each sequence, the
    tokens to compute (None = all).  Yields (packed rows, o, bound) per
    sequence, o (rows, Hq, D)."""
    G, a = q.shape[1] // k.shape[1], 0
    for n in lens:
        if n:
            t = torch.arange(n, device=q.device) if rows_of is None else rows_of(n).to(q.device)
            see = torch.arange(n, device=q.device) <= t[:, None]
            os, bs = [], []
            for h in range(q.shape[1]):
                o, b = rows(q[a + t, h].double(), k[a:a + n, h // G].double(), v[a:a + n, h // G].double(), see, scale)
                os.append(o)
                bs.append(b)
            yield a + t, torch.stack(os, 1), torch.stack(bs, 1)
        a += n


def tree(q, k, v, nodes, mask, kc, vc, table, ctx, scale):
    """attn_tree: kc, vc (pages, page, Hkv, D); a page outside the cache is zeros."""
    G, a, page = q.shape[1] // k.shape[1], 0, kc.shape[1]
    dev = q.device
    for b, (n, c) in enumerate(zip(nodes, ctx)):
        if n:
            j = torch.arange(c, device=dev)
            pg = table[b].long()[j // page] if c else j
            ok = (pg >= 0) & (pg < kc.shape[0])
            pg = torch.where(ok, pg, torch.zeros_like(pg))
            words = mask[a:a + n].tolist()
            new = torch.tensor([[w >> i & 1 for i in range(n)] for w in words], dtype=torch.bool, device=dev)
            see = torch.cat([torch.ones(n, c, dtype=torch.bool, device=dev), new], 1)
            os, bs = [], []
            for h in range(q.shape[1]):
                hk = h // G
                ks = torch.cat([torch.where(ok[:, None], kc[pg, j % page, hk], 0), k[a:a + n, hk]]).double()
                vs = torch.cat([torch.where(ok[:, None], vc[pg, j % page, hk], 0), v[a:a + n, hk]]).double()
                # an unseen key's own values have no part in any row
                dead = ~see.any(0)
                o, bd = rows(q[a:a + n, h].double(), torch.where(dead[:, None], 0.0, ks), vs, see, scale)
                os.append(o)
                bs.append(bd)
            yield torch.arange(a, a + n, device=dev), torch.stack(os, 1), torch.stack(bs, 1)
        a += n


def norm_rope(x, w, eps, cos_sin, pos, inter):
    """qk_norm_rope of one tensor (T, H, D) in 64 bits, and how far the fp32
    value may be from it before it is rounded to bf16: sums of D squares and
    three products, 2^-16 of the rotated pair's magnitudes."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    z, mag = y.clone(), y.abs()
    if cos_sin is not None and cos_sin.shape[1]:
        rot = cos_sin.shape[1]
        half = rot // 2
        cs = cos_sin.double()[pos.long()][:, None]
        i = torch.arange(half, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + half)
        a, b, c, s = y[..., ia], y[..., ib], cs[..., :half], cs[..., half:]
        z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return z, 2.0 ** -16 * mag + 1e-38


def assert_rounded(got, want, off, what):
    """got is the bf16 rounding of a value within off of want (NaN where want is)."""
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all()), f"{what}: NaN in other places than the definition's"
    out = ~nan & ((got < (want - off).to(torch.bfloat16)) | (got > (want + off).to(torch.bfloat16)))
    if bool(out.any()):
        i = tuple(int(x) for x in out.nonzero()[0])
        raise AssertionError(f"{what}: {int(out.sum())} of {out.numel()} values are not the rounding of a value within "
                             f"their bound, first at {i}: got {float(got[i])}, want {float(want[i])} +- {float(off[i])}")


def assert_within(got, want, bound, what):
    got = got.double()
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all()), f"{what}: NaN in other places than the definition's"
    over = torch.where(nan, torch.zeros_like(want), (got - want).abs() - bound)
    worst = float(over.max()) if over.numel() else 0.0
    if worst > 0:
        i = tuple(int(x) for x in (over == over.max()).nonzero()[0])
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} values past their bound, worst at {i}: "
                             f"got {float(got[i])}, want {float(want[i])} +- {float(bound[i])}")

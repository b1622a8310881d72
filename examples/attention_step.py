"""The attention sublayer of a draft layer, prompt pass and verify step, with
the package's quantized linears around the attention operators:

    qkv = FP8 PTPC GEMM       fp8_quantize_act, fp8_gemm_ptpc
    q, k normed and rotated   qk_norm_rope (a prompt's k and v into the cache)
    attention                 attn_prompt | attn_tree over the paged cache
    o = MXFP4 A4W4 GEMM       mx_gemm_a4w4 with bf16 activations
    the accepted path         kv_append

Run it: python examples/attention_step.py   (a GB300 and the built library)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_dynamic_gb300 as mx  # noqa: E402


def rope_table(positions: int, rot: int, device) -> torch.Tensor:
    """(positions, rot) f32, a row [cos | sin], angles in 64 bits."""
    p = torch.arange(positions, dtype=torch.float64)
    a = p[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


class Attention:
    """Weights of one attention sublayer and its paged cache."""

    def __init__(self, hidden=7168, hq=64, hkv=8, d=128, pages=256, page_size=64, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, sigma: (torch.randn(*s, generator=g) * sigma).bfloat16().to(device)  # noqa: E731
        self.hq, self.hkv, self.d, self.hidden, self.page_size = hq, hkv, d, hidden, page_size
        self.wqkv, self.sqkv = mx.fp8_quantize_weight(rnd((hq + 2 * hkv) * d, hidden, sigma=0.02), layout=mx.PANEL)
        self.wo, _ = mx.mx_quantize_weight(rnd(hidden, hq * d, sigma=0.02), layout=mx.PANEL)
        self.wq, self.wk = (1 + rnd(d, sigma=0.1).float()).bfloat16(), (1 + rnd(d, sigma=0.1).float()).bfloat16()
        self.cos_sin = rope_table(4096, d, device)
        shape = (pages, page_size, hkv, d)
        self.cache = mx.KVCache(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                                torch.zeros(shape, dtype=torch.bfloat16, device=device))

    def _qkv(self, x, pos, **cache):
        """q, k (normed and rotated, in place) and v of hidden states x (T, hidden)."""
        qa, sa = mx.fp8_quantize_act(x)
        y = mx.fp8_gemm_ptpc(qa, sa, self.wqkv, self.sqkv, weights_tiled=mx.W_PANEL, k=self.hidden)
        y = y.view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = y[:, :self.hq], y[:, self.hq:self.hq + self.hkv], y[:, self.hq + self.hkv:]
        mx.qk_norm_rope(q, k, pos, self.cos_sin, wq=self.wq, wk=self.wk, q_out=q, k_out=k,
                        v=v if cache else None, **cache)
        return q, k, v

    def _o(self, a):
        return mx.mx_gemm_a4w4(self.wo, None, x=a.view(-1, self.hq * self.d), weights_tiled=mx.W_PANEL, n=self.hidden,
                               k=self.hq * self.d)

    def prompt(self, x, pos, cu, slots):
        """A prompt pass of packed sequences; k and v go into the cache.
        Returns (o_proj's output, the attention's)."""
        q, k, v = self._qkv(x, pos, cache=self.cache, slots=slots)
        a = mx.attn_prompt(q, k, v, cu)
        return self._o(a), a

    def verify(self, x, pos, cu, mask, table, ctx):
        """A verify step over trees of drafted tokens.  Returns (o_proj's
        output, the attention's, k, v): what is accepted of k and v goes to
        accept()."""
        q, k, v = self._qkv(x, pos)
        a = mx.attn_tree(q, k, v, cu, mask, self.cache, table, ctx)
        return self._o(a), a, k, v

    def accept(self, k, v, cu, path, table, ctx):
        return mx.kv_append(k, v, cu, path, self.cache, table, ctx)


def run(hidden=7168, hq=64, hkv=8, d=128, lens=(300, 45, 1024), seed=1, device="cuda"):
    """Prompts, one verify step of a tree a sequence, the accepted path into
    the cache, one more token -- and the same tokens as one prompt.  Returns
    the last token's attention both ways, (sequences, hq, d) each."""
    layer = Attention(hidden, hq, hkv, d, seed=seed, device=device)
    g = torch.Generator().manual_seed(seed + 1)
    B, page = len(lens), layer.page_size
    # a page table with room for the prompt and what is accepted
    need = [(n + 8) // page + 1 for n in lens]
    order = torch.randperm(256, generator=g).tolist()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    x = [torch.randn(n, hidden, generator=g).bfloat16() for n in lens]
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(device)
    slots = torch.cat([table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
                       for b, n in enumerate(lens)]).to(device)
    cu = ints([0] + torch.tensor(lens).cumsum(0).tolist())
    layer.prompt(torch.cat(x).to(device), pos, cu, slots)
    # a tree a sequence: the verified token, two tries for the next, three below the second
    depth, up, path = [0, 1, 1, 2, 2, 3], [-1, 0, 0, 2, 2, 4], [0, 2, 4, 5]
    see = []
    for i, u in enumerate(up):
        see.append((see[u] if u >= 0 else 0) | 1 << i)
    t = [torch.randn(len(up), hidden, generator=g).bfloat16() for _ in lens]
    ctx, table = ints(lens), table.to(device)
    cn = ints([len(up) * b for b in range(B + 1)])
    tpos = torch.cat([n + torch.tensor(depth) for n in lens]).int().to(device)
    mask = torch.tensor(see * B, dtype=torch.int64, device=device)
    _, _, k, v = layer.verify(torch.cat(t).to(device), tpos, cn, mask, table, ctx)
    ctx = layer.accept(k, v, cn, ints([path + [-1]] * B), table, ctx)
    # one more token: a tree of one node
    last = [torch.randn(1, hidden, generator=g).bfloat16() for _ in lens]
    _, got, _, _ = layer.verify(torch.cat(last).to(device), ctx.clone(), ints(list(range(B + 1))),
                                torch.ones(B, dtype=torch.int64, device=device), table, ctx)
    # the same tokens as prompts
    whole = [torch.cat([x[b], t[b][path], last[b]]) for b in range(B)]
    n = [len(w) for w in whole]
    _, a = layer.prompt(torch.cat(whole).to(device), torch.cat([torch.arange(m) for m in n]).int().to(device),
                        ints([0] + torch.tensor(n).cumsum(0).tolist()),
                        torch.full((sum(n),), -1, dtype=torch.int64, device=device))
    want = a[torch.tensor(n).cumsum(0).to(device) - 1]
    return got, want


if __name__ == "__main__":
    got, want = run()
    torch.cuda.synchronize()
    off = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"token after prompt, verified tree and accepted path: {tuple(got.shape)}, "
          f"relative difference from the same tokens as one prompt {off:.2e}")

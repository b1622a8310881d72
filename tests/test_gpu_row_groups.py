"""attn_shared and attn_sparse where heads of a kv head do not divide a tile's 128 rows: a row group has 2 floor(128 / G)
nodes, and a record's last one counts however many records a call has (32 are counted by the kernel itself)."""
import pytest
import torch

import attn_ref
import test_gpu_attn_shared as shared
import test_gpu_attn_sparse as sparse
import fp8_block_scaled_dynamic_gb300 as mx

pytestmark = pytest.mark.gpu


def nan_like(t):
    return torch.full_like(t, float("nan"))


def nan_bytes(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


SHARED = [
    # one launch, more than 32 records; the prefix's row groups
    ([38], [256], [8] * 38, 40, 8),
    ([39], [128], [13] * 39, 24, 8),
    ([41], [192], [8] * 41, 96, 8),
    # and the sequences' own
    ([], [], [51] * 33, 20, 4),
    ([33], [64], [21, 63, 41, 62] * 8 + [1], 12, 1),
    ([], [], [25, 49, 50] * 12, 10, 1),
    ([], [], [23] * 17 + [45, 46] * 9, 11, 1),
    ([], [], [19] * 17 + [37, 38, 55, 56, 57] * 4, 13, 1),
    # two launches, more than 32 groups
    ([51] + [1] * 40, [64] * 41, [1] * 91, 40, 8),
    ([102, 3] + [2] * 33, [128, 64] + [64] * 33, [1] * 171, 5, 1),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("i", range(len(SHARED)))
def test_shared(D, i):
    groups, prefix, nodes, Hq, Hkv = SHARED[i]
    c = shared.Case(groups, prefix, [17 * b % 150 for b in range(len(nodes))], nodes, Hq, Hkv, D, 64, seed=50 + i)
    ws = nan_bytes(mx.mxg_attn_shared_workspace_bytes(sum(nodes), Hq, D))
    c.check(c.run(out=nan_like(c.q), ws=ws), SHARED[i][2:])


def check_lists(c, out, what):
    """Of every row what its lists name, in 64 bits."""
    G, page, a = c.q.shape[1] // c.k.shape[1], c.kc.shape[1], 0
    for b, (n, ctx) in enumerate(zip(c.nodes, c.ctx)):
        j = torch.arange(ctx, device=c.q.device)
        pages, words = c.tab[b].long()[j // page], c.mask[a:a + n].tolist()
        new = torch.tensor([[w >> i & 1 for i in range(n)] for w in words], dtype=torch.bool, device=c.q.device)
        for h in range(c.k.shape[1]):
            see = torch.cat([((j // page)[None, :, None] == c.sel[a:a + n, h, None].long()).any(-1), new], 1)
            ks = torch.cat([c.kc[pages, j % page, h], c.k[a:a + n, h]]).double()
            vs = torch.cat([c.vc[pages, j % page, h], c.v[a:a + n, h]]).double()
            for g in range(h * G, h * G + G):
                o, bound = attn_ref.rows(c.q[a:a + n, g].double(), ks, vs, see, c.scale)
                attn_ref.assert_within(out[a:a + n, g], o, bound, f"{what}: sequence {b} head {g}")
        a += n


SPARSE = [
    ([51] * 5, 40, 8), ([21] * 5, 96, 8), ([63] * 5, 96, 8), ([25] * 5, 80, 8), ([50, 49, 25, 24, 50] * 4, 20, 2),
    ([23, 45, 46, 22, 44] * 7, 11, 1), ([19, 37, 38, 55, 56, 57] * 3, 26, 2), ([64, 42, 43] * 12, 3, 1),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("i", range(len(SPARSE)))
def test_sparse(D, i):
    nodes, Hq, Hkv = SPARSE[i]
    c = sparse.Case([200 + 37 * b % 230 for b in range(len(nodes))], nodes, Hq, Hkv, D, 32, 4, seed=70 + i)
    ws = nan_bytes(mx.mxg_attn_sparse_workspace_bytes(sum(nodes), Hkv, 4, D))
    check_lists(c, c.run(out=nan_like(c.q), ws=ws), SPARSE[i])

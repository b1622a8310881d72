"""attn_prompt against softmax attention in 64 bits."""
import math

import pytest
import torch

import attn_ref
import fp8_block_scaled_dynamic_gb300 as mx
from gpu_util import dev

pytestmark = pytest.mark.gpu


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def offsets(lens, d):
    return torch.tensor([0] + list(lens)).cumsum(0).int().to(d)


def inputs(seed, T, Hq, Hkv, D, d):
    return (randn(seed, T, Hq, D, scale=1.5).to(d), randn(seed + 1, T, Hkv, D).to(d), randn(seed + 2, T, Hkv, D).to(d))


def check(out, q, k, v, lens, scale, what, rows_of=None):
    for at, o, b in attn_ref.prompt(q, k, v, lens, scale, rows_of):
        attn_ref.assert_within(out[at], o, b, what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([1], 8, 1), ([1, 0, 1, 2], 4, 4), ([127], 2, 2), ([128], 2, 1), ([129], 3, 1), ([16, 17, 15, 33], 16, 2),
    ([0, 255, 256, 257, 0], 8, 8), ([700, 3, 130], 10, 2), ([513], 14, 2), ([300], 7, 1), ([90, 41], 71, 1),
    ([50, 140], 128, 1), ([260, 1], 130, 2), ([1000], 12, 4),
])
def test_prompt(D, lens, Hq, Hkv):
    d = dev()
    T = sum(lens)
    q, k, v = inputs(T + Hq, T, Hq, Hkv, D, d)
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    check(out, q, k, v, lens, 1 / math.sqrt(D), f"{lens} {Hq}/{Hkv} D={D}")


def test_prompt_long_sampled_rows():
    """One long sequence and a short one: rows at tile edges and at random."""
    d = dev()
    lens, Hq, Hkv, D = [5003, 260], 8, 2, 128
    q, k, v = inputs(1, sum(lens), Hq, Hkv, D, d)
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    g = torch.Generator().manual_seed(2)
    check(out, q, k, v, lens, 1 / math.sqrt(D), "long", lambda n: torch.unique(torch.cat(
        [torch.tensor([0, 1, 31, 32, 127, 128, 129, n - 2, n - 1]), torch.randint(0, n, (60,), generator=g)])))


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_strides(D):
    """Slices of a packed projection, and tensors laid out head by head."""
    d = dev()
    lens, Hq, Hkv = [70, 200], 6, 2
    T = sum(lens)
    qkv = randn(3, T, Hq + 2 * Hkv, D).to(d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = mx.attn_prompt(q, k, v, offsets(lens, d), scale=0.2)
    check(out, q, k, v, lens, 0.2, "packed")
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    o2 = torch.empty(Hq, T, D, dtype=torch.bfloat16, device=d).transpose(0, 1)
    mx.attn_prompt(*hm, offsets(lens, d), scale=0.2, out=o2)
    assert torch.equal(o2, out)


def test_prompt_tokens_past_the_last_sequence_are_not_written():
    d = dev()
    lens, T = [40, 100], 200
    q, k, v = inputs(5, T, 4, 2, 64, d)
    k[140:], v[140:] = float("nan"), float("nan")
    out = torch.full_like(q, 7.0)
    mx.attn_prompt(q, k, v, offsets(lens, d), out=out)
    check(out, q[:140], k[:140], v[:140], lens, 1 / 8, "front")
    assert bool((out[140:] == 7.0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_special_values_reach_only_those_who_see_them(D, bad):
    """k and v of one token are NaN or infinite in some channels: earlier
    tokens and other sequences are as if it were not there."""
    d = dev()
    lens, Hq, Hkv = [100, 300, 50], 8, 2
    T = sum(lens)
    q, k, v = inputs(6, T, Hq, Hkv, D, d)
    ref = mx.attn_prompt(q, k, v, offsets(lens, d))
    at = 100 + 165
    v[at, 0, 3] = bad
    v[at, 1, D - 1] = bad
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    sees = torch.zeros(T, dtype=torch.bool, device=d)
    sees[at:400] = True
    assert torch.equal(out[~sees], ref[~sees])
    hit = torch.zeros(T, Hq, D, dtype=torch.bool, device=d)
    hit[at:400, :4, 3] = True
    hit[at:400, 4:, D - 1] = True
    assert not bool(torch.isfinite(out[hit]).any()) and bool(torch.isfinite(out[~hit]).all())
    v[at] = 0
    k[at, 0, 5] = float("nan")
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    assert bool(torch.isnan(out[at:400, :4]).all()) and bool(torch.isfinite(out[:, 4:]).all())
    assert torch.equal(out[~sees], ref[~sees])


def test_prompt_large_scores():
    """Scores far apart: the running maximum moves by much, the weights of the
    others vanish, nothing overflows."""
    d = dev()
    lens, Hq, Hkv, D = [600], 4, 2, 128
    q, k, v = inputs(8, 600, Hq, Hkv, D, d)
    k *= (1 + torch.arange(600, device=d) % 97)[:, None, None].bfloat16()
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    check(out, q, k, v, lens, 1 / math.sqrt(D), "spread")
    k = k[torch.arange(599, -1, -1, device=d)] * 50
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    assert bool(torch.isfinite(out).all())


def test_prompt_repeats_and_streams():
    d = dev()
    lens = [300, 17, 640]
    q, k, v = inputs(9, sum(lens), 8, 2, 128, d)
    cu = offsets(lens, d)
    want = mx.attn_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [mx.attn_prompt(q, k, v, cu, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=d)
    assert mx.attn_prompt(e, e, e, offsets([0, 0], d)).shape == (0, 8, 128)


def test_prompt_many_sequences():
    d = dev()
    g = torch.Generator().manual_seed(10)
    lens = torch.randint(0, 9, (1500,), generator=g).tolist()
    lens[700] = 400
    T = sum(lens)
    q, k, v = inputs(11, T, 2, 1, 64, d)
    out = mx.attn_prompt(q, k, v, offsets(lens, d))
    check(out, q, k, v, lens, 1 / 8, "many")


def test_prompt_offsets_out_of_range_are_clamped():
    d = dev()
    q, k, v = inputs(12, 50, 2, 1, 64, d)
    cu = torch.tensor([0, 30, 10, 90], dtype=torch.int32, device=d)   # falls, then runs past T
    out = torch.zeros_like(q)
    mx.attn_prompt(q, k, v, cu, out=out)
    assert bool(torch.isfinite(out).all())
    check(out, q[:30], k[:30], v[:30], [30], 1 / 8, "first")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([1], 8, 1), ([300], 7, 1), ([0, 255, 256, 257, 0], 8, 8), ([700, 3, 130], 64, 8), ([513], 14, 2), ([90, 41], 71, 1),
    ([1100, 600], 32, 16),
])
def test_prompt_is_the_same_in_a_larger_batch(D, lens, Hq, Hkv):
    """However the rows are grouped (a batch of more than 32 sequences, a few
    long or short ones), a row's result is the same, and within the bound; so
    is what a NaN reaches."""
    d = dev()
    T = sum(lens)
    q, k, v = inputs(20 + T, T, Hq, Hkv, D, d)
    cu = offsets(lens, d)
    many = torch.cat([torch.zeros(20, dtype=torch.int32, device=d), cu, cu[-1:].expand(20)])
    out = mx.attn_prompt(q, k, v, many)
    check(out, q, k, v, lens, 1 / math.sqrt(D), f"{lens} {Hq}/{Hkv} D={D}, 40 empty sequences more")
    assert torch.equal(mx.attn_prompt(q, k, v, cu), out)
    longest = max(range(len(lens)), key=lambda b: lens[b])
    at = sum(lens[:longest]) + lens[longest] // 2
    v[at, 0, 1] = float("nan")
    a, b = mx.attn_prompt(q, k, v, many), mx.attn_prompt(q, k, v, cu)
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    sees = torch.zeros(T, Hq, D, dtype=torch.bool, device=d)
    sees[at:sum(lens[:longest + 1]), :Hq // Hkv, 1] = True
    assert bool(a[sees].isnan().all()) and torch.equal(a[~sees], out[~sees])

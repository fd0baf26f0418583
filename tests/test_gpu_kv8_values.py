"""Attention over the int8 cache where its value is decided by few bits or by the ends of the
range: value scales, queries, weights and tables that the sums in 64 bits see and a rounding at
the wrong place does not.  Every test runs in each tile height: 4, 8, 16 and 32 query rows."""
import math

import pytest
import torch

from test_gpu_kv8 import BLOCK, attend, ints, page_table, random_cache, whole

pytestmark = pytest.mark.gpu

# queries, query heads, cache heads: rows of a tile 4, 8, 16, 32
HEIGHTS = [(1, 2, 1), (1, 8, 1), (4, 4, 1), (8, 4, 1), (33, 2, 2)]


def scales_of(cache, t, table, j):
    """View of the scales [heads] of a sequence's block j."""
    page = cache[t + "_codes"].shape[2]
    return cache[t + "_scale"][int(table[j * BLOCK // page]), :, j * BLOCK % page // BLOCK]


def codes_of(cache, t, table, j):
    page = cache[t + "_codes"].shape[2]
    at = j * BLOCK % page
    return cache[t + "_codes"][int(table[j * BLOCK // page]), :, at:at + BLOCK]


def in_64_bits(q, n, table, cache, causal, scale):
    """(weights p [m][heads][n], scores, values [heads][n][D], sizes of the scores) of one
    sequence, for every query head."""
    Hq, Hkv = q.shape[1], cache["k_codes"].shape[1]
    k = whole(cache["k_codes"], cache["k_scale"], table, n).repeat_interleave(Hq // Hkv, 0)
    v = whole(cache["v_codes"], cache["v_scale"], table, n).repeat_interleave(Hq // Hkv, 0)
    s = torch.einsum("mhd,hnd->mhn", q.double(), k) * scale
    size = torch.einsum("mhd,hnd->mhn", q.double().abs(), k.abs()) * abs(scale)
    if causal:
        m = q.shape[0]
        hidden = torch.arange(n, device="cuda")[None] > \
            n - m + torch.arange(m, device="cuda")[:, None]
        s = s.masked_fill(hidden[:, None], -math.inf)
        size = size.masked_fill(hidden[:, None], 0)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-300), s, v, size


def check(out, want, spread, held, relative):
    """out within half a bf16 step of want, `relative` of spread = sum p|v| and `held`."""
    allow = want.abs() * 2.0 ** -8 + spread * relative + held
    off = (out.double() - want).abs()
    assert bool((off <= allow).all()), float((off / allow).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", HEIGHTS)
@pytest.mark.parametrize("far", [0, 1, 9, 70])
@pytest.mark.parametrize("causal", [False, True])
def test_a_block_without_weight_takes_no_bits(causal, far, m, Hq, Hkv, D):
    """Block `far` has a value scale 2^45 above the others' and scores that leave it no weight
    (or, causal, the last token lies behind what the earlier queries see and has it): the
    other blocks' values come out as if it were not there.  Allowed: weights of 11 bits,
    2^-36 of the row's largest p * scale * 127 for each token, scores off by 2^-22 of their size
    in (D / 16 + 8) steps, sums over the blocks in fp32."""
    n, page, scale = 1200, 32, 0.125
    table, pages = page_table([n], page, seed=far)
    cache = random_cache(pages, Hkv, page, D, far + D)
    g = torch.Generator(device="cuda").manual_seed(far + m)
    q = torch.randn(m, Hq, D, generator=g, device="cuda").bfloat16()
    q[..., 0] = 4.0
    for j in range(-(-n // BLOCK)):
        codes_of(cache, "k", table[0], j)[..., 0] = 0
    last = -(-n // BLOCK) - 1
    far = last if causal else far
    scales_of(cache, "v", table[0], far).mul_(2.0 ** 45)
    if not causal:
        codes_of(cache, "k", table[0], far)[..., 0] = -127
        scales_of(cache, "k", table[0], far).fill_(4.0)
        codes_of(cache, "k", table[0], far)[..., 1:] = 0
    out, _ = attend(q, ints([0, m]), ints([n]), table, cache, causal, scale)
    p, s, v, size = in_64_bits(q, n, table[0], cache, causal, scale)
    spread = torch.einsum("mhn,hnd->mhd", p, v.abs())
    block_max = v.abs().amax(-1).view(Hq, -1, BLOCK).amax(-1).repeat_interleave(BLOCK, 1)
    held = (p * block_max).amax(-1, keepdim=True) * n * 2.0 ** -36
    steps = float(size.max() + 1) * (D / 16 + 8) * 2.0 ** -22
    check(out, torch.einsum("mhn,hnd->mhd", p, v), spread, held,
          2.0 ** -11 + 2 * steps + (n / BLOCK + 32) * 2.0 ** -22)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", HEIGHTS)
@pytest.mark.parametrize("n", [1, 40])
def test_small_values_of_a_query_beside_a_large_one(n, m, Hq, Hkv, D):
    """One channel of q is 2^13, and its key codes are 0: the scores are those of the other
    channels.  Allowed: values below 2^-21 of the row's largest off by 2^-30 of it; the sum of
    digits or of (D / 16 + 8) steps in fp32, 2^-22 of the terms' sizes each; the logarithm's
    result, 2^-22 of it."""
    page, scale = 16, 0.125
    table, pages = page_table([n], page)
    cache = random_cache(pages, Hkv, page, D, n + D)
    cache["k_codes"][..., 5] = 0
    g = torch.Generator(device="cuda").manual_seed(m + n)
    q = torch.randn(m, Hq, D, generator=g, device="cuda").bfloat16()
    q[..., 5] = 8192.0
    _, lse = attend(q, ints([0, m]), ints([n]), table, cache, False, scale)
    _, s, _, size = in_64_bits(q, n, table[0], cache, False, scale)
    k = whole(cache["k_codes"], cache["k_scale"], table[0], n).repeat_interleave(Hq // Hkv, 0)
    small = (q.double().abs() < 2.0 ** -8).double() * 2.0 ** -17
    held = torch.einsum("mhd,hnd->mhn", small, k.abs()).amax(-1) * scale
    want = torch.logsumexp(s, -1)
    allow = held + (size.amax(-1) + 1) * (D / 16 + 8) * 2.0 ** -22 + want.abs() * 2.0 ** -22
    off = (lse.double() - want).abs()
    assert bool((off <= allow).all()), float((off / allow).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", HEIGHTS)
@pytest.mark.parametrize("n", [2, 16, 24])
def test_weights_of_values_that_cancel(n, m, Hq, Hkv, D):
    """Neighbouring tokens have opposite values and keys that differ by a code: what is left is
    the difference of weights about 2^-12 apart, which 11 bits do not have.  Allowed: weights
    held to 2^-22 and their largest's 2^-35; scores off by 2^-22 of their size in (D / 16 + 8)
    steps, twice (the weight and the sum that divides it); sums over the blocks in fp32."""
    page, scale = 16, 0.125
    table, pages = page_table([n], page)
    cache = random_cache(pages, Hkv, page, D, n + D)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    k, v = cache["k_codes"], cache["v_codes"]
    k.clamp_(-126, 126)
    step = torch.randint(-1, 2, k[:, :, 1::2].shape, generator=g, device="cuda", dtype=torch.int8)
    k[:, :, 1::2] = k[:, :, 0::2] + step
    v[:, :, 1::2] = -v[:, :, 0::2]
    q = (torch.randn(m, Hq, D, generator=g, device="cuda") * 0.02).bfloat16()
    out, _ = attend(q, ints([0, m]), ints([n]), table, cache, False, scale)
    p, s, v8, size = in_64_bits(q, n, table[0], cache, False, scale)
    steps = float(size.max() + 1) * (D / 16 + 8) * 2.0 ** -22
    check(out, torch.einsum("mhn,hnd->mhd", p, v8), torch.einsum("mhn,hnd->mhd", p, v8.abs()), 0,
          2.0 ** -22 + n * 2.0 ** -35 + 2 * steps + (n / BLOCK + 32) * 2.0 ** -22)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", HEIGHTS)
@pytest.mark.parametrize("n", [30, 3000])
@pytest.mark.parametrize("size", [2.0 ** 119, 2.0 ** -124])
def test_values_at_the_ends_of_the_range(size, n, m, Hq, Hkv, D):
    """Values up to 1.2 * 2^126 and down to 2^-131: their means are in range.  Allowed: half a
    bf16 step, 2^-22 of sum p|v| as for any other values (weights, scores, sums), and the
    ends' own steps: 2^-134 for bf16, 2^-135 for sums of p v over each part of the tokens."""
    page, scale = 64, 0.125
    table, pages = page_table([n], page)
    cache = random_cache(pages, Hkv, page, D, n + D)
    cache["v_scale"].fill_(size)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    q = torch.randn(m, Hq, D, generator=g, device="cuda").bfloat16()
    out, _ = attend(q, ints([0, m]), ints([n]), table, cache, True, scale)
    p, s, v8, sizes = in_64_bits(q, n, table[0], cache, True, scale)
    steps = float(sizes.max() + 1) * (D / 16 + 8) * 2.0 ** -22
    check(out, torch.einsum("mhn,hnd->mhd", p, v8), torch.einsum("mhn,hnd->mhd", p, v8.abs()),
          2.0 ** -134 + n / BLOCK * 2.0 ** -135,
          2.0 ** -22 + n * 2.0 ** -35 + 2 * steps + (n / BLOCK + 32) * 2.0 ** -22)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", HEIGHTS)
@pytest.mark.parametrize("n", [3, 100, 5000])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_is_seen(bad, n, m, Hq, Hkv, D):
    """One value of one query and head is not finite, in a channel whose key codes are 0: all of
    its results are NaN (zeros and -infinity if it sees no token), all others are as before."""
    page, scale = 32, 0.125
    table, pages = page_table([n], page)
    cache = random_cache(pages, Hkv, page, D, n)
    cache["k_codes"][..., 9] = 0
    g = torch.Generator(device="cuda").manual_seed(m + n)
    q = torch.randn(m, Hq, D, generator=g, device="cuda").bfloat16()
    for i in {0, m - 1}:
        x = q.clone()
        calm = attend(x, ints([0, m]), ints([n]), table, cache, True, scale)
        x[i, 1, 9] = bad
        out, lse = attend(x, ints([0, m]), ints([n]), table, cache, True, scale)
        if n - m + i >= 0:
            assert bool(out[i, 1].isnan().all()) and bool(lse[i, 1].isnan())
        else:
            assert bool((out[i, 1] == 0).all()) and float(lse[i, 1]) == -math.inf
        out[i, 1], lse[i, 1] = calm[0][i, 1], calm[1][i, 1]
        assert torch.equal(out, calm[0]) and torch.equal(lse, calm[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv", [(4, 1, 1), (8, 1, 1), (16, 1, 1), (20, 4, 1), (40, 2, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("t", ["k", "v"])
def test_scales_of_blocks_that_a_query_does_not_see(t, bad, m, Hq, Hkv, D):
    """Causal, and the last block's scale is not finite: the queries that do not see it have what
    they have without it, bit for bit; those that do are not finite."""
    page, scale = 16, 0.125
    for n in (33, 97, 417):                                # one token in the last block
        table, pages = page_table([n], page)
        cache = random_cache(pages, Hkv, page, D, n)
        g = torch.Generator(device="cuda").manual_seed(m + n)
        q = torch.randn(m, Hq, D, generator=g, device="cuda").bfloat16()
        out, lse = attend(q, ints([0, m]), ints([n]), table, cache, True, scale)
        scales_of(cache, t, table[0], n // BLOCK).fill_(bad)
        bad_out, bad_lse = attend(q, ints([0, m]), ints([n]), table, cache, True, scale)
        assert torch.equal(bad_out[:-1], out[:-1]) and torch.equal(bad_lse[:-1], lse[:-1])
        assert not bool(bad_out[-1].isfinite().any())

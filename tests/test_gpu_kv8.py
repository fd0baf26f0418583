"""The paged int8 cache: appended codes and scales bit for bit against numpy, attention
over the cache against 64-bit sums, and a decoding step of both with the weight-only
products around them."""
import math

import numpy as np
import pytest
import torch

import activation_quantized_gemm_wq_b200 as wq

pytestmark = pytest.mark.gpu

BLOCK = 16


def page_table(lens, page, extra=3, seed=0, width=None):
    need = [-(-n // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(need) + extra)
    table = np.full((len(lens), width or max(1, max(need, default=1))), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), sum(need) + extra


def starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def random_cache(pages, heads, page, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = {}
    for t in ("k", "v"):
        c[t + "_codes"] = torch.randint(-127, 128, (pages, heads, page, D), generator=g,
                                        device="cuda", dtype=torch.int8)
        c[t + "_scale"] = torch.rand(pages, heads, page // BLOCK, generator=g, device="cuda") \
            * 0.02 + 0.005
    return c


# ---------------------------------------------------------------- append

def append_reference(x, row_start, past, table, codes, scale):
    """One of keys / values, in IEEE fp32 (numpy): codes and scale are changed in place."""
    page_tokens = codes.shape[2]
    for b in range(len(past)):
        r, end, p = row_start[b], row_start[b + 1], past[b]
        while r < end:
            inside = p % BLOCK
            n = min(BLOCK - inside, end - r)
            page, slot = table[b, p // page_tokens], p % page_tokens - inside
            for h in range(codes.shape[1]):
                rows = x[r:r + n, h]
                blk = codes[page, h, slot:slot + BLOCK]
                old = scale[page, h, slot // BLOCK] if inside else np.float32(0)
                s = max(old, np.float32(np.abs(rows).max()) / np.float32(127))
                if inside and s > old:
                    blk[:inside] = np.rint(blk[:inside].astype(np.float32) * (old / s))
                with np.errstate(divide="ignore", invalid="ignore"):
                    q = np.clip(np.rint(rows / s), -127, 127) if s > 0 else np.zeros_like(rows)
                blk[inside:inside + n] = q
                scale[page, h, slot // BLOCK] = s
            r, p = r + n, p + n


def run_append(new, past, heads, D, page, size=1.0, seed=0):
    """Appends on the GPU and in the reference; returns both caches as numpy."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    T = sum(new)
    qkv = (torch.randn(T, 3, heads, D, generator=g, device="cuda") * size).bfloat16()
    qkv *= torch.exp(torch.randn(T, 1, 1, 1, generator=g, device="cuda") * 0.7)
    k, v = qkv[:, 1], qkv[:, 2]
    table, pages = page_table([a + b for a, b in zip(new, past)], page, seed=seed)
    cache = random_cache(pages, heads, page, D, seed)
    want = {n: t.cpu().numpy().copy() for n, t in cache.items()}
    start = starts(new)
    wq.wq_kv8_append(k, v, start, ints(past), table, **cache)
    for t, x in (("k", k), ("v", v)):
        append_reference(x.float().cpu().numpy(), start.tolist(), past, table.cpu().numpy(),
                         want[t + "_codes"], want[t + "_scale"])
    return {n: t.cpu().numpy() for n, t in cache.items()}, want


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("new,past", [
    ([1], [0]), ([1, 1, 1, 1], [5, 16, 127, 128]), ([3, 0, 40, 1], [15, 9, 0, 200]),
    ([300], [7]), ([16, 16], [0, 8]), ([0, 0, 17], [3, 0, 31]), ([130, 90], [64, 63])])
def test_append_is_bit_exact(new, past, page, D):
    got, want = run_append(new, past, 3, D, page, seed=len(new) + page)
    for n in want:
        assert np.array_equal(got[n], want[n]), n
    assert wq.wq_device_status() == ("WQ_OK", 0)


@pytest.mark.parametrize("size", [0.0, 1e-39, 1e-36, 1e35])
def test_append_at_the_ends_of_the_range(size):
    """Zeros (scale 0, codes 0), subnormal values and scales, large ones."""
    got, want = run_append([20, 1], [3, 16], 2, 64, 32, size=size, seed=5)
    for n in want:
        assert np.array_equal(got[n], want[n]), n


def test_append_token_by_token_keeps_the_largest_scale_and_bounded_codes():
    """Tokens one call at a time: each block's scale is the one that a single call gives,
    and a value is off by at most half a step for its own rounding and half a step of the
    then larger scale for each of the 15 tokens that may follow."""
    D, heads, n = 64, 2, 37
    x = torch.randn(n, heads, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    table, pages = page_table([n], 16)
    one, many = random_cache(pages, heads, 16, D, 1), random_cache(pages, heads, 16, D, 2)
    wq.wq_kv8_append(x, x, ints([0, n]), ints([0]), table, **one)
    for i in range(n):
        wq.wq_kv8_append(x[i:i + 1], x[i:i + 1], ints([0, 1]), ints([i]), table, **many)
    at = table[0].long()
    used = (n + 15) // 16
    assert torch.equal(one["k_scale"][at[:used]], many["k_scale"][at[:used]])
    c = many["k_codes"][at].permute(1, 0, 2, 3).reshape(heads, -1, D)[:, :n].double()
    s = many["k_scale"][at].permute(1, 0, 2).reshape(heads, -1).repeat_interleave(16, 1)[:, :n]
    off = (c * s[..., None].double() - x.permute(1, 0, 2).double()).abs() / s[..., None].double()
    assert float(off.max()) <= 0.5 + 15 * 0.5 + 1e-3
    assert float(off.pow(2).mean().sqrt()) < 1.0


def test_append_leaves_other_rows_and_sequences_alone():
    """Rows outside [row_start[0], row_start[B]) are not read (NaN there), sequences that
    do not fit and bad pages are not written and reported, the others are done."""
    D, heads, page = 64, 2, 32
    table, pages = page_table([64, 64, 64], page, seed=4)
    table[1, 0] = pages                                       # outside the cache
    cache = random_cache(pages, heads, page, D, 6)
    want = {n: t.cpu().numpy().copy() for n, t in cache.items()}
    x = torch.randn(80, heads, D, device="cuda").bfloat16()
    x[:5] = float("nan")
    x[70:] = float("nan")
    start = ints([5, 25, 35, 70])
    past = [3, 0, 30]                                         # the third: 30 + 35 > 64
    wq.wq_kv8_append(x, x, start, ints(past), table, **cache)
    for t in ("k", "v"):
        append_reference(x.float().cpu().numpy(), [5, 25], past[:1], table.cpu().numpy(),
                         want[t + "_codes"], want[t + "_scale"])
    for n in want:
        assert np.array_equal(cache[n].cpu().numpy(), want[n]), n
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)
    assert wq.wq_device_status() == ("WQ_OK", 0)


@pytest.mark.parametrize("starts_bad", [[0, 5, 3, 8], [0, 4, 9], [-2, 4, 8]])
def test_append_reports_bad_row_tables(starts_bad):
    """Rows that go back, end behind T or begin before 0: reported, nothing out of bounds."""
    D, heads, page, B = 64, 1, 16, len(starts_bad) - 1
    table, pages = page_table([32] * B, page)
    cache = random_cache(pages, heads, page, D, 6)
    x = torch.randn(8, heads, D, device="cuda").bfloat16()
    wq.wq_kv8_append(x, x, ints(starts_bad), ints([0] * B), table, **cache)
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)


# ---------------------------------------------------------------- attention

def whole(codes, scale, table_row, n):
    """Cached values [heads][n][D] of one sequence in 64 bits."""
    page = codes.shape[2]
    at = table_row[:-(-n // page)].long()
    c = codes[at].double() * scale[at].double().repeat_interleave(BLOCK, 2)[..., None]
    return c.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def check_attention(q, q_lens, kv_lens, table, cache, causal, scale, out, lse, first=0):
    """out and lse against 64-bit sums.  One rounding of out to bf16 (2^-8 of it); for the
    sums of p v, in units of sum p|v| / sum p: the weights' rounding to f16 (2^-11, and
    those below 2^-25 of the largest, steps of 2^-35 of it, by at most 2^-36), scores in fp32 (products
    exact, D / 16 matrix steps, two scalings and the exponential's 2^-22, each relative to
    the sum of magnitudes), and fp32 additions over the blocks."""
    Hq, D = q.shape[1:]
    r = first
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        Hkv = cache["k_codes"].shape[1]
        G = Hq // Hkv
        for h in range(Hkv if m else 0):
            rows = slice(r, r + m)
            got_o, got_l = out[rows, h * G:h * G + G].double(), lse[rows, h * G:h * G + G].double()
            if n == 0:
                assert bool((got_o == 0).all()) and bool((got_l == -math.inf).all())
                continue
            k = whole(cache["k_codes"], cache["k_scale"], table[b], n)[h]
            v = whole(cache["v_codes"], cache["v_scale"], table[b], n)[h]
            x = q[rows, h * G:h * G + G].double()
            s = torch.einsum("mgd,nd->mgn", x, k) * scale
            size = torch.einsum("mgd,nd->mgn", x.abs(), k.abs()).amax(-1) * abs(scale)
            if causal:
                hidden = torch.arange(n, device="cuda")[None] > \
                    n - m + torch.arange(m, device="cuda")[:, None]
                s = s.masked_fill(hidden[:, None], -math.inf)
            want_l = torch.logsumexp(s, -1)
            empty = want_l == -math.inf
            p = torch.exp(s - want_l.masked_fill(empty, 0)[..., None])
            want_o = p @ v
            spread = p @ v.abs()
            per_score = (D / 16 + 8) * 2.0 ** -22 * (size + 1)
            sums = (n / BLOCK + 32) * 2.0 ** -22
            allow = want_o.abs() * 2.0 ** -8 + spread * (2.0 ** -11 + 2 * per_score + sums
                                                         )[..., None] + 2.0 ** -24 * v.abs().max()
            assert bool((got_o[empty] == 0).all()) and bool((got_l[empty] == -math.inf).all())
            assert bool(((got_o - want_o).abs() <= allow).all())
            off = (got_l - want_l).abs()[~empty]
            assert bool((off <= (per_score + sums + want_l.abs() * 2.0 ** -22)[~empty]).all())
        r += m
    return r


def attend(q, q_start, kv_len, table, cache, causal, scale, out=None, lse=None, ws=None, **kw):
    Tq, Hq, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    out = torch.full((Tq, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((Tq, Hq), 7.0, device="cuda") if lse is None else lse
    ws = wq.alloc_attn_workspace(Tq, kv_len.shape[0], Hq, Hkv, D) if ws is None else ws
    wq.wq_attn_kv8(q, q_start, kv_len, table, cache["k_codes"], cache["v_codes"],
                   cache["k_scale"], cache["v_scale"], causal, scale, out, lse, ws, **kw)
    return out, lse


def run_attention(q_lens, kv_lens, Hq, Hkv, D, page, causal, seed=0, q_size=1.5, extra_rows=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 17)
    table, pages = page_table(kv_lens, page, seed=seed)
    cache = random_cache(pages, Hkv, page, D, seed)
    T = sum(q_lens) + extra_rows
    q = (torch.randn(T, Hq, D, generator=g, device="cuda") * q_size).bfloat16()
    scale = D ** -0.5
    out, lse = attend(q, starts(q_lens), ints(kv_lens), table, cache, causal, scale)
    rows = check_attention(q, q_lens, kv_lens, table, cache, causal, scale, out, lse)
    assert bool((out[rows:] == 7).all()) and bool((lse[rows:] == 7).all())
    assert wq.wq_device_status() == ("WQ_OK", 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,page", [
    ([1], [1], 1, 1, 16), ([1], [15], 2, 2, 16), ([1], [16], 4, 1, 32), ([1], [17], 8, 2, 64),
    ([1], [129], 3, 3, 128), ([1, 1, 1], [0, 33, 700], 5, 1, 16), ([1], [5000], 16, 2, 64),
    ([1] * 40, [37 * i + 1 for i in range(40)], 8, 8, 32),
    ([1, 1], [4097, 2], 32, 2, 16), ([7], [100], 6, 2, 32), ([2, 0, 5], [64, 50, 31], 9, 3, 16),
    ([20], [20], 2, 1, 16), ([33, 64], [40, 1000], 4, 4, 64), ([64], [700], 12, 4, 32),
    ([100, 3, 1], [2000, 3, 900], 7, 7, 128), ([9, 9], [4, 0], 2, 2, 16),
    ([257], [300], 4, 2, 16), ([1], [40000], 2, 1, 128)])
def test_attention(q_lens, kv_lens, Hq, Hkv, page, causal, D):
    run_attention(q_lens, kv_lens, Hq, Hkv, D, page, causal, seed=sum(kv_lens) % 1000)


def test_attention_of_many_short_sequences():
    """More sequences than threads in a CTA, several without queries or without a cache."""
    r = np.random.RandomState(3)
    q_lens = [int(v) for v in r.randint(0, 3, 400)]
    kv_lens = [int(v) for v in r.randint(0, 90, 400)]
    run_attention(q_lens, kv_lens, 4, 2, 64, 16, False, seed=9)
    run_attention(q_lens, kv_lens, 4, 2, 64, 16, True, seed=10, extra_rows=6)


@pytest.mark.parametrize("q_size", [0.0, 1e-30, 30.0, 1e6])
def test_attention_with_small_and_large_queries(q_size):
    """Flat softmax, one-hot softmax; queries outside f16's range."""
    run_attention([1, 4], [333, 90], 4, 2, 64, 32, True, seed=2, q_size=q_size)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
@pytest.mark.parametrize("m,Hq,Hkv", [(1, 4, 2), (1, 8, 1), (3, 4, 1), (30, 2, 2)])
def test_attention_scales(scale, m, Hq, Hkv):
    """Negative, zero and large softmax scales, in every tile height."""
    n, D, page = 700, 64, 32
    table, pages = page_table([n], page, seed=2)
    cache = random_cache(pages, Hkv, page, D, 8)
    q = torch.randn(m, Hq, D, generator=torch.Generator(device="cuda").manual_seed(4),
                    device="cuda").bfloat16()
    out, lse = attend(q, ints([0, m]), ints([n]), table, cache, True, scale)
    check_attention(q, [m], [n], table, cache, True, scale, out, lse)


def test_attention_rising_scores_and_uneven_value_scales():
    """The running maximum moves in every block, and value blocks differ in scale by 2^20,
    among them zero scales: the sums are rescaled again and again."""
    D, n, page = 128, 2000, 64
    table, pages = page_table([n], page, seed=1)
    cache = random_cache(pages, 1, page, D, 3)
    at = table[0].long()
    for j in range(-(-n // BLOCK)):
        blk = cache["k_codes"][at[j * BLOCK // page], 0, j * BLOCK % page:j * BLOCK % page + BLOCK]
        blk.fill_(min(127, j))
        cache["k_scale"][at[j * BLOCK // page], 0, j * BLOCK % page // BLOCK] = 0.05
        cache["v_scale"][at[j * BLOCK // page], 0, j * BLOCK % page // BLOCK] = \
            0.0 if j % 5 == 4 else 2.0 ** ((j * 7) % 21 - 10)
    q = torch.full((1, 2, D), 0.25, dtype=torch.bfloat16, device="cuda")
    q[0, 1] = -0.25
    out, lse = attend(q, ints([0, 1]), ints([n]), table, cache, True, 1.0)
    check_attention(q, [1], [n], table, cache, True, 1.0, out, lse)


def test_attention_ignores_what_lies_behind_the_sequence():
    """Slots behind kv_len, pages that no table names and table entries behind the last
    page may hold anything, NaN scales among it."""
    D, page, n = 64, 32, 41
    table, pages = page_table([n], page, extra=4, width=5)
    cache = random_cache(pages, 2, page, D, 1)
    q = torch.randn(1, 2, D, device="cuda").bfloat16()
    out, lse = attend(q, ints([0, 1]), ints([n]), table, cache, False, 0.125)
    used = table[0, :2].long()
    for t in ("k", "v"):
        spare = torch.ones(pages, dtype=torch.bool, device="cuda")
        spare[used] = False
        cache[t + "_scale"][spare] = float("nan")
        cache[t + "_scale"][used[1], :, 1] = float("nan")     # tokens 48 to 63
        cache[t + "_codes"][used[1], :, 9:] = -128
    again, lse2 = attend(q, ints([0, 1]), ints([n]), table, cache, False, 0.125)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert wq.wq_device_status() == ("WQ_OK", 0)


def test_attention_reports_bad_tables_and_stays_in_bounds():
    D, page = 64, 16
    table, pages = page_table([32, 32], page)
    cache = random_cache(pages, 1, page, D, 1)
    q = torch.randn(2, 1, D, device="cuda").bfloat16()
    good, _ = attend(q, ints([0, 1, 2]), ints([32, 32]), table, cache, False, 0.125)
    for table2, kv in ((table.clone(), [32, 32]), (table, [-5, 32]), (table, [33, 32])):
        if table2 is not table:
            table2[0, 1] = -1
        out, _ = attend(q, ints([0, 1, 2]), ints(kv), table2, cache, False, 0.125)
        assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)
        assert torch.equal(out[1], good[1])
    out, _ = attend(q, ints([0, 1, 9]), ints([32, 32]), table, cache, False, 0.125)
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)
    out, _ = attend(q, ints([0, 1, 2]), ints([32, 32]), table, cache, False, 0.125)
    assert torch.equal(out, good) and wq.wq_device_status() == ("WQ_OK", 0)


def test_attention_on_strided_queries_and_without_lse():
    """q as a part of a fused projection's rows, no lse, another stream."""
    D, H, page = 128, 4, 32
    table, pages = page_table([300], page)
    cache = random_cache(pages, H, page, D, 4)
    qkv = torch.randn(5, 3, H, D, device="cuda").bfloat16()
    q = qkv[:, 0]
    out, lse = attend(q, ints([0, 5]), ints([300]), table, cache, True, 0.09)
    check_attention(q, [5], [300], table, cache, True, 0.09, out, lse)
    plain, _ = attend(q.contiguous(), ints([0, 5]), ints([300]), table, cache, True, 0.09)
    assert torch.equal(out, plain)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = torch.zeros_like(out)
    ws = wq.alloc_attn_workspace(5, 1, H, H, D)
    args = (q, ints([0, 5]), ints([300]), table, cache["k_codes"], cache["v_codes"],
            cache["k_scale"], cache["v_scale"], True, 0.09, other, None, ws)
    torch.cuda.synchronize()
    wq.wq_attn_kv8(*args, stream=side)
    side.synchronize()
    assert torch.equal(out, other)


def test_attention_on_two_streams_at_once_and_repeated():
    """Two calls that overlap, each with a workspace of its own, and the same call many
    times: the same bits."""
    D, page = 128, 64
    lens = [3000, 10, 900]
    table, pages = page_table(lens, page)
    cache = random_cache(pages, 2, page, D, 4)
    q = torch.randn(3, 8, D, device="cuda").bfloat16()
    start, kv = ints([0, 1, 2, 3]), ints(lens)
    want, want_l = attend(q, start, kv, table, cache, True, 0.09)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in range(2)]
    lses = [torch.zeros_like(want_l) for _ in range(2)]
    wss = [wq.alloc_attn_workspace(3, 3, 8, 2, D) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            attend(q, start, kv, table, cache, True, 0.09, outs[i], lses[i], wss[i],
                   stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want) and torch.equal(lses[i], want_l)


def test_attention_beyond_two_gib_of_codes():
    """Pages whose byte offset passes 2^31 (and 2^32 over both arrays)."""
    D, page, heads = 128, 128, 8
    pages = (1 << 31) // (page * heads * D) + 40
    cache = {t + "_codes": torch.zeros(pages, heads, page, D, dtype=torch.int8, device="cuda")
             for t in ("k", "v")}
    cache |= {t + "_scale": torch.zeros(pages, heads, page // BLOCK, device="cuda")
              for t in ("k", "v")}
    n = 1000
    table = ints([[pages - 1 - i for i in range(8)]])
    x = torch.randn(n, heads, D, generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda").bfloat16()
    wq.wq_kv8_append(x, -x, ints([0, n]), ints([0]), table, **cache)
    assert int((cache["k_codes"][:pages - 8] != 0).sum()) == 0
    q = torch.randn(1, 16, D, device="cuda").bfloat16()
    out, lse = attend(q, ints([0, 1]), ints([n]), table, cache, True, 0.09)
    check_attention(q, [1], [n], table, cache, True, 0.09, out, lse)
    assert wq.wq_device_status() == ("WQ_OK", 0)


# ---------------------------------------------------------------- together

def test_decoding_steps_in_one_graph():
    """The q/k/v product, append, attention and the output product of a small layer, three
    sequences, captured once and replayed token by token with lengths that move on the
    device; each step is checked against the state it started from."""
    B, H, D, K, group, page, steps = 3, 4, 64, 256, 64, 16, 20
    g = torch.Generator(device="cuda").manual_seed(11)
    past0 = [0, 13, 90]
    table, pages = page_table([p + steps for p in past0], page)
    cache = random_cache(pages, H, page, D, 2)

    def layer(n, k):
        W = (torch.randn(n, k, generator=g, device="cuda") * 0.1).bfloat16()
        qw = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
        s_g = torch.empty(k // group, n, dtype=torch.bfloat16, device="cuda")
        wq.wq_pack_int4_group(W, None, group, qw, s_g)
        return qw, s_g

    w_in, w_out = layer(3 * H * D, K), layer(K, H * D)
    x = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(B, 3, H, D, dtype=torch.bfloat16, device="cuda")
    att, lse = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, device="cuda")
    y = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
    start, past, kv = ints([0, 1, 2, 3]), ints(past0), ints([p + 1 for p in past0])
    ws = wq.alloc_attn_workspace(B, B, H, H, D)

    def step():
        wq.wq_gemv_w4g(x, None, *w_in, group, None, qkv.view(B, -1))
        wq.wq_kv8_append(qkv[:, 1], qkv[:, 2], start, past, table, **cache)
        wq.wq_attn_kv8(qkv[:, 0], start, kv, table, cache["k_codes"], cache["v_codes"],
                       cache["k_scale"], cache["v_scale"], True, D ** -0.5, att, lse, ws)
        wq.wq_gemv_w4g(att.view(B, -1), None, *w_out, group, None, y)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    from test_gpu_group import check_gemv
    for i in range(steps):
        x.copy_(torch.randn(B, K, generator=g, device="cuda"))
        before = {n: t.cpu().numpy().copy() for n, t in cache.items()}
        graph.replay()
        torch.cuda.synchronize()
        check_gemv(x, None, *w_in, group, None, qkv.view(B, -1))
        for j, t in ((1, "k"), (2, "v")):
            append_reference(qkv[:, j].float().cpu().numpy(), [0, 1, 2, 3], past.tolist(),
                             table.cpu().numpy(), before[t + "_codes"], before[t + "_scale"])
        for n in before:
            assert np.array_equal(cache[n].cpu().numpy(), before[n], equal_nan=True), n
        check_attention(qkv[:, 0], [1] * B, kv.tolist(), table, cache, True, D ** -0.5, att, lse)
        check_gemv(att.view(B, -1), None, *w_out, group, None, y)
        past += 1
        kv += 1
    assert wq.wq_device_status() == ("WQ_OK", 0)

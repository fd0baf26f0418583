"""The int8 cache's device checks: every table that the header forbids is reported, whichever
rows the calls' warps look at, and a good one is not."""
import numpy as np
import pytest
import torch

import activation_quantized_gemm_wq_b200 as wq
from test_gpu_kv8 import append_reference, attend, ints, page_table, random_cache

pytestmark = pytest.mark.gpu

T, D, HEADS, PAGE, ROOM = 8, 64, 2, 16, 32      # rows, head size, heads, page and table sizes

# row_start, past_len: 8 rows, room for 32 tokens in each sequence's table
BAD = [([0, 8, 9], [0, 0]), ([9, 12], [0]), ([8, 9], [0]), ([-3, 0, 8], [0, 0]), ([-3, -1], [0]),
       ([0, 8, 8], [0, -1]), ([0, 0, 8], [-5, 0]), ([8, 8], [-1]), ([0, 8, 8], [0, 33]),
       ([0, 4, 2, 8], [0, 0, 0]), ([0, 8], [25]), ([0, 8, 2147483647], [0, 0]),
       ([-2147483648, 0, 8], [0, 0]), ([0, 8], [2147483647]), ([0, 8, 8], [0, -2147483648])]
GOOD = [([0, 8, 8], [0, 32]), ([0, 8], [24]), ([3, 3, 5], [32, 30]), ([8, 8], [0])]


def append(starts, past):
    table, pages = page_table([ROOM] * len(past), PAGE)
    cache = random_cache(pages, HEADS, PAGE, D, 6)
    before = {n: t.clone() for n, t in cache.items()}
    x = torch.randn(T, HEADS, D, generator=torch.Generator(device="cuda").manual_seed(1),
                    device="cuda").bfloat16()
    wq.wq_kv8_append(x, x, ints(starts), ints(past), table, **cache)
    return x, table, cache, before


@pytest.mark.parametrize("starts,past", BAD)
def test_append_reports_every_bad_table(starts, past):
    """Reported, and a sequence whose rows lie within T and fit is written as if alone."""
    x, table, cache, before = append(starts, past)
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)
    if starts == sorted(starts):
        want = {n: t.cpu().numpy().copy() for n, t in before.items()}
        for b, p in enumerate(past):
            lo, hi = starts[b:b + 2]
            if lo < 0 or hi > T or p < 0 or p + hi - lo > ROOM:
                continue
            for t in ("k", "v"):
                append_reference(x.float().cpu().numpy(), [lo, hi], [p], table[b:b + 1].cpu().numpy(),
                                 want[t + "_codes"], want[t + "_scale"])
        for n in want:
            assert np.array_equal(cache[n].cpu().numpy(), want[n]), n


@pytest.mark.parametrize("starts,past", GOOD)
def test_append_reports_no_good_table(starts, past):
    append(starts, past)
    assert wq.wq_device_status() == ("WQ_OK", 0)


def test_append_looks_at_every_one_of_many_sequences():
    """The only bad entry is the last of 1000 sequences, without rows."""
    n = 1000
    table = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    cache = random_cache(3, HEADS, PAGE, D, 6)
    x = torch.randn(T, HEADS, D, device="cuda").bfloat16()
    starts, past = [0] + [T] * n, [0] * n
    wq.wq_kv8_append(x, x, ints(starts), ints(past), table, **cache)
    assert wq.wq_device_status() == ("WQ_OK", 0)
    past[-1] = -1
    wq.wq_kv8_append(x, x, ints(starts), ints(past), table, **cache)
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)


@pytest.mark.parametrize("starts,past", BAD)
def test_attention_reports_every_bad_table(starts, past):
    """The same tables as queries' rows and cached lengths."""
    table, pages = page_table([ROOM] * len(past), PAGE)
    cache = random_cache(pages, HEADS, PAGE, D, 6)
    q = torch.randn(T, HEADS, D, device="cuda").bfloat16()
    attend(q, ints(starts), ints([p + 8 if p == 25 else p for p in past]), table, cache, False, 0.1)
    assert wq.wq_device_status() == ("WQ_ERR_DEVICE", 4)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("t", ["k", "v"])
def test_append_of_a_value_that_is_not_finite_is_seen(t, bad, D):
    """Its block of its head has a scale that is NaN, also after more tokens came to the block,
    until a sequence begins it anew; the other blocks and heads, and of keys and values the
    other one, are what they are without it."""
    page, n, at = 32, 40, 21                               # token 21 lies in block 1
    table, pages = page_table([64], page)
    g = torch.Generator(device="cuda").manual_seed(D)
    x = {u: torch.randn(64, HEADS, D, generator=g, device="cuda").bfloat16() for u in "kv"}
    y = {u: x[u].clone() for u in "kv"}
    y[t][at, 1, 5] = bad
    good, got = random_cache(pages, HEADS, page, D, 2), random_cache(pages, HEADS, page, D, 2)
    for cache, rows in ((good, x), (got, y)):
        for lo, hi in ((0, 18), (18, 30), (30, n)):        # block 1: begun, gone on with, ended
            wq.wq_kv8_append(rows["k"][lo:hi], rows["v"][lo:hi], ints([0, hi - lo]), ints([lo]),
                             table, **cache)
    hit = int(table[0, 0])
    assert bool(got[t + "_scale"][hit, 1, 1].isnan())
    q = torch.randn(1, HEADS, D, device="cuda").bfloat16()
    out, lse = attend(q, ints([0, 1]), ints([n]), table, got, True, 0.1)
    want, want_lse = attend(q, ints([0, 1]), ints([n]), table, good, True, 0.1)
    assert bool(out[0, 1].isnan().all()) and torch.equal(out[0, 0], want[0, 0])
    assert bool(lse[0, 1].isnan()) == (t == "k") and torch.equal(lse[0, 0], want_lse[0, 0])
    for u in "kv":
        for kind in ("_codes", "_scale"):
            a, b = got[u + kind].clone(), good[u + kind].clone()
            if u == t:
                blk = (hit, 1, slice(16, 32)) if kind == "_codes" else (hit, 1, 1)
                a[blk], b[blk] = 0, 0
            assert torch.equal(a, b), u + kind
    wq.wq_kv8_append(x["k"][:n], x["v"][:n], ints([0, n]), ints([0]), table, **got)
    assert bool(got[t + "_scale"][hit, 1, 1].isfinite())
    assert wq.wq_device_status() == ("WQ_OK", 0)


def test_both_error_words_are_read_and_cleared_together():
    """A stream id outside the table and a bad row table, then neither."""
    table, pages = page_table([ROOM], PAGE)
    cache = random_cache(pages, HEADS, PAGE, D, 6)
    x = torch.randn(T, HEADS, D, device="cuda").bfloat16()
    K = HEADS * D
    ids = torch.tensor([0] * (T - 1) + [5], dtype=torch.uint8, device="cuda")
    quantized = (torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"))

    def quantize(stream_id):
        wq.wq_act_quant(x.view(T, K), torch.ones(K, device="cuda"), stream_id,
                        torch.ones(1, 3, device="cuda"), 0, 8, *quantized)

    for rows, stream_id, flags in (([9, 12], ids, 6), ([0, 8], ids, 2), ([9, 12], ids * 0, 4)):
        wq.wq_kv8_append(x, x, ints(rows), ints([0]), table, **cache)
        quantize(stream_id)
        assert wq.wq_device_status() == ("WQ_ERR_DEVICE", flags)
        assert wq.wq_device_status() == ("WQ_OK", 0)

"""The group-scaled weights' and the int8 cache's entry points refuse bad arguments on the
host, before any launch: the library by its status codes, the binding by looking at the
tensors.  No GPU: addresses are made up and never followed."""
import ctypes

import pytest
import torch

import activation_quantized_gemm_wq_b200 as wq
from activation_quantized_gemm_wq_b200 import build as wq_build
from test_binding_checks import DevT, fake  # noqa: F401

FAKE = 1 << 20
BF16, F32, I32, I8, U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8)


@pytest.fixture(scope="module")
def lib():
    if wq_build.needs_build():
        wq_build.build()
    return wq.lib()


def at(n):
    return FAKE + n


def _pack(lib, **kw):
    a = dict(W=FAKE, c=FAKE, N=16, K=256, group=64, qw=FAKE, s_g=FAKE) | kw
    return lib.wq_pack_int4_group(a["W"], a["c"], a["N"], a["K"], a["group"], a["qw"], a["s_g"],
                                  None)


@pytest.mark.parametrize("kw,code", [
    (dict(group=16), 4), (dict(group=0), 4), (dict(group=256), 4), (dict(K=200), 2),
    (dict(K=65536), 2), (dict(N=0), 2), (dict(N=2147483647, K=32768), 2), (dict(W=None), 1),
    (dict(qw=None), 1), (dict(s_g=None), 1), (dict(W=at(8)), 3), (dict(c=at(4)), 3),
    (dict(qw=at(8)), 3), (dict(s_g=at(1)), 3)])
def test_pack_refuses(lib, kw, code):
    assert _pack(lib, **kw) == code


def _gemv(lib, **kw):
    a = dict(x=FAKE, M=4, K=256, N=16, cinv=FAKE, qw=FAKE, s_g=FAKE, group=64, bias=FAKE,
             y=FAKE) | kw
    return lib.wq_gemv_w4g(a["x"], a["M"], a["K"], a["N"], a["cinv"], a["qw"], a["s_g"],
                           a["group"], a["bias"], a["y"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(group=48), 4), (dict(K=100), 2), (dict(M=-1), 2), (dict(M=17), 2), (dict(N=0), 2),
    (dict(N=2147483647), 2), (dict(x=None), 1), (dict(qw=None), 1), (dict(s_g=None), 1),
    (dict(y=None), 1), (dict(x=at(2)), 3), (dict(qw=at(4)), 3), (dict(s_g=at(1)), 3),
    (dict(y=at(1)), 3), (dict(bias=at(2)), 3), (dict(cinv=at(8)), 3),
    (dict(M=0, x=None, y=None), 0)])
def test_gemv_refuses(lib, kw, code):
    assert _gemv(lib, **kw) == code


CACHE = dict(B=2, max_pages=4, pages=9, heads=2, page=32, D=64)


def _append(lib, **kw):
    a = CACHE | dict(k=FAKE, v=FAKE, ks=128, vs=128, T=5, start=FAKE, past=FAKE, table=FAKE,
                     kc=FAKE, vc=FAKE, s_k=FAKE, s_v=FAKE) | kw
    return lib.wq_kv8_append(a["k"], a["v"], a["ks"], a["vs"], a["T"], a["start"], a["past"],
                             a["B"], a["table"], a["max_pages"], a["kc"], a["vc"], a["s_k"],
                             a["s_v"], a["pages"], a["heads"], a["page"], a["D"], None)


BAD_CACHE = [
    (dict(B=-1), 2), (dict(max_pages=0), 2), (dict(pages=0), 2), (dict(heads=0), 2),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(D=96), 2), (dict(D=256), 2),
    (dict(pages=1 << 26), 2),               # pages * heads * page_tokens = 2^32
    (dict(max_pages=1 << 26), 2),           # 2^31 token positions
    (dict(start=None), 1), (dict(table=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(s_k=None), 1), (dict(s_v=None), 1), (dict(start=at(2)), 3), (dict(table=at(2)), 3),
    (dict(kc=at(8)), 3), (dict(vc=at(8)), 3), (dict(s_k=at(2)), 3), (dict(s_v=at(1)), 3)]


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(T=-1), 2), (dict(ks=120), 2), (dict(vs=132), 2), (dict(ks=0), 2), (dict(ks=-128), 2),
    (dict(T=2000000000, heads=64, ks=4096, vs=4096), 2), (dict(k=None), 1), (dict(v=None), 1),
    (dict(past=None), 1), (dict(k=at(8)), 3), (dict(v=at(2)), 3), (dict(past=at(1)), 3),
    (dict(T=0, k=None, v=None), 0), (dict(B=0, table=None), 0)])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code


def _attn(lib, **kw):
    a = CACHE | dict(q=FAKE, qs=256, Tq=5, Hq=4, start=FAKE, kv=FAKE, table=FAKE, kc=FAKE,
                     vc=FAKE, s_k=FAKE, s_v=FAKE, causal=1, scale=0.125, out=FAKE, lse=None,
                     ws=FAKE, n=1 << 40) | kw
    return lib.wq_attn_kv8(a["q"], a["qs"], a["Tq"], a["Hq"], a["start"], a["kv"], a["B"],
                           a["table"], a["max_pages"], a["kc"], a["vc"], a["s_k"], a["s_v"],
                           a["pages"], a["heads"], a["page"], a["D"], a["causal"], a["scale"],
                           a["out"], a["lse"], a["ws"], ctypes.c_size_t(a["n"]), None)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(Tq=-1), 2), (dict(Hq=3), 2), (dict(Hq=0), 2), (dict(qs=255), 2), (dict(qs=248), 2),
    (dict(Tq=1 << 30), 2), (dict(scale=float("nan")), 4), (dict(scale=float("inf")), 4),
    (dict(q=None), 1), (dict(kv=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(q=at(8)), 3), (dict(out=at(8)), 3), (dict(kv=at(2)), 3), (dict(lse=at(2)), 3),
    (dict(ws=at(16)), 3), (dict(n=0), 4), (dict(Tq=0, q=None, out=None, ws=None, n=0), 0),
    (dict(B=0, table=None, ws=None, n=0), 0)])
def test_attention_refuses(lib, kw, code):
    assert _attn(lib, **kw) == code


def test_attention_workspace(lib):
    n = wq.wq_attn_kv8_workspace_bytes(5, 2, 4, 2, 64)
    assert n > 0 and n % 256 == 0
    assert _attn(lib, n=n - 1) == 4
    # more rows per sequence: larger tiles; invalid sizes: none
    assert wq.wq_attn_kv8_workspace_bytes(64, 2, 4, 2, 64) > n
    for bad in ((5, 2, 3, 2, 64), (5, 2, 4, 2, 80), (-1, 2, 4, 2, 64), (5, -1, 4, 2, 64),
                (5, 2, 4, 0, 64)):
        assert wq.wq_attn_kv8_workspace_bytes(*bad) == 0
    with pytest.raises(ValueError):
        wq.alloc_attn_workspace(5, 2, 3, 2, 64)


# ---------------------------------------------------------------- the binding

class RowT(DevT):
    """DevT with strides of its own."""
    def __init__(self, shape, dtype, strides=None, **kw):
        super().__init__(shape, dtype, **kw)
        self._s = strides or self._t.stride()

    def stride(self):
        return self._s


M, K, N, G = 3, 256, 24, 64


def weights():
    return dict(W=RowT((N, K), BF16), c=RowT((K,), F32), x=RowT((M, K), BF16),
                cinv=RowT((K,), F32), qw=RowT((N, K // 2), U8), s_g=RowT((K // G, N), BF16),
                bias=RowT((N,), F32), y=RowT((M, N), BF16))


def test_group_wrappers_marshal_in_header_order(fake):  # noqa: F811
    a = weights()
    wq.wq_pack_int4_group(a["W"], a["c"], G, a["qw"], a["s_g"], stream=0)
    wq.wq_gemv_w4g(a["x"], a["cinv"], a["qw"], a["s_g"], G, a["bias"], a["y"], stream=0)
    p = {n: t.addr for n, t in a.items()}
    assert fake.calls == [
        ("wq_pack_int4_group", (p["W"], p["c"], N, K, G, p["qw"], p["s_g"], 0)),
        ("wq_gemv_w4g", (p["x"], M, K, N, p["cinv"], p["qw"], p["s_g"], G, p["bias"], p["y"], 0))]


@pytest.mark.parametrize("key,bad", [
    ("x", RowT((M, K), F32)), ("x", RowT((M, K), BF16, cuda=False)),
    ("x", RowT((M, K), BF16, contiguous=False)), ("x", RowT((M, K), BF16, device=1)),
    ("cinv", RowT((K - 1,), F32)), ("qw", RowT((N, K // 2 - 1), U8)),
    ("qw", RowT((N, K // 2), I32)), ("s_g", RowT((K // G - 1, N), BF16)),
    ("s_g", RowT((K // G, N), F32)), ("bias", RowT((N - 1,), F32)), ("y", RowT((M, N - 1), BF16)),
    ("y", RowT((M, N), F32))])
def test_gemv_wrapper_refuses_a_bad_tensor(fake, key, bad):  # noqa: F811
    a = weights() | {key: bad}
    with pytest.raises((ValueError, TypeError)):
        wq.wq_gemv_w4g(a["x"], a["cinv"], a["qw"], a["s_g"], G, a["bias"], a["y"], stream=0)
    assert fake.calls == []


@pytest.mark.parametrize("key,bad", [
    ("c", RowT((K - 1,), F32)), ("qw", RowT((N - 1, K // 2), U8)),
    ("s_g", RowT((K // G, N - 1), BF16)), ("s_g", RowT((K // G, N), F32)), ("W", RowT((N, K), F32))])
def test_pack_wrapper_refuses_a_bad_tensor(fake, key, bad):  # noqa: F811
    a = weights() | {key: bad}
    with pytest.raises((ValueError, TypeError)):
        wq.wq_pack_int4_group(a["W"], a["c"], G, a["qw"], a["s_g"], stream=0)
    assert fake.calls == []


B, T, H, HQ, D, P, PAGES, MAXP = 2, 5, 2, 4, 64, 32, 7, 3


def cached():
    qkv = (HQ + 2 * H) * D     # rows of a fused projection
    return dict(q=RowT((T, HQ, D), BF16, (qkv, D, 1)), k=RowT((T, H, D), BF16, (qkv, D, 1)),
                v=RowT((T, H, D), BF16), start=RowT((B + 1,), I32), past=RowT((B,), I32),
                kv=RowT((B,), I32), table=RowT((B, MAXP), I32), kc=RowT((PAGES, H, P, D), I8),
                vc=RowT((PAGES, H, P, D), I8), s_k=RowT((PAGES, H, P // 16), F32),
                s_v=RowT((PAGES, H, P // 16), F32), out=RowT((T, HQ, D), BF16),
                lse=RowT((T, HQ), F32), ws=RowT((4096,), U8))


def _w_append(a):
    wq.wq_kv8_append(a["k"], a["v"], a["start"], a["past"], a["table"], a["kc"], a["vc"],
                     a["s_k"], a["s_v"], stream=0)


def _w_attn(a):
    wq.wq_attn_kv8(a["q"], a["start"], a["kv"], a["table"], a["kc"], a["vc"], a["s_k"], a["s_v"],
                   True, 0.125, a["out"], a["lse"], a["ws"], stream=0)


def test_cache_wrappers_marshal_in_header_order(fake):  # noqa: F811
    a = cached()
    _w_append(a)
    _w_attn(a)
    p = {n: t.addr for n, t in a.items()}
    wide = (HQ + 2 * H) * D
    assert fake.calls == [
        ("wq_kv8_append", (p["k"], p["v"], wide, H * D, T, p["start"], p["past"], B, p["table"],
                           MAXP, p["kc"], p["vc"], p["s_k"], p["s_v"], PAGES, H, P, D, 0)),
        ("wq_attn_kv8", (p["q"], wide, T, HQ, p["start"], p["kv"], B, p["table"], MAXP, p["kc"],
                         p["vc"], p["s_k"], p["s_v"], PAGES, H, P, D, 1, 0.125, p["out"],
                         p["lse"], p["ws"], 4096, 0))]


BAD_TENSORS = [
    ("table", RowT((B + 1, MAXP), I32)), ("table", RowT((B * MAXP,), I32)),
    ("table", RowT((B, MAXP), torch.int64)), ("kc", RowT((PAGES, H, P, D), U8)),
    ("vc", RowT((PAGES - 1, H, P, D), I8)), ("vc", RowT((PAGES, H, P, D), I8, contiguous=False)),
    ("s_k", RowT((PAGES, H, P // 32), F32)), ("s_v", RowT((PAGES, H, P // 16), BF16)),
    ("start", RowT((B,), I32)), ("start", RowT((B + 1,), torch.int64))]


@pytest.mark.parametrize("key,bad", BAD_TENSORS + [
    ("k", RowT((T, H, D + 1), BF16)), ("k", RowT((T, H + 1, D), BF16)), ("k", RowT((T, H * D), BF16)),
    ("k", RowT((T, H, D), BF16, (H * D, 1, H))), ("v", RowT((T, H, D), F32)),
    ("v", RowT((T + 1, H, D), BF16)), ("v", RowT((T, H, D), BF16, cuda=False)),
    ("v", RowT((T, H, D), BF16, device=1))])
def test_append_wrapper_refuses_a_bad_tensor(fake, key, bad):  # noqa: F811
    with pytest.raises((ValueError, TypeError)):
        _w_append(cached() | {key: bad})
    assert fake.calls == []


@pytest.mark.parametrize("key,bad", BAD_TENSORS + [
    ("q", RowT((T, HQ, D // 2), BF16)), ("q", RowT((T, HQ, D), BF16, (HQ * D, D, 2))),
    ("q", RowT((T, HQ, D), torch.float16)), ("out", RowT((T, HQ, D - 1), BF16)),
    ("out", RowT((T, HQ, D), F32)), ("lse", RowT((T, HQ - 1), F32)), ("lse", RowT((T, HQ), BF16)),
    ("out", RowT((T, HQ, D), BF16, contiguous=False))])
def test_attention_wrapper_refuses_a_bad_tensor(fake, key, bad):  # noqa: F811
    with pytest.raises((ValueError, TypeError)):
        _w_attn(cached() | {key: bad})
    assert fake.calls == []

"""Cases for the low-bit operators that serve one denoising or decoding step beside the
fused linears: weight-only matrix-vector products with int4 codes and group scales, and
attention over a paged int8 key/value cache with a scale per block of 16 tokens and head.

  pack    wq_pack_int4_group   weights -> int4 codes and one bf16 scale per group of channels
  gemv    wq_gemv_w4g          1 to 16 tokens times such weights
  append  wq_kv8_append        new keys and values quantized into the cache's pages
  attn    wq_attn_kv8          attention of some queries over the cache

With own = False every operator is computed from its formula with elementary torch
operations in fp32 and rounded once at the end; with own = True by the library's kernels.
Both work on the same packed weights, pages and tables."""
import math
import random

import torch

own = False

BLOCK = 16     # tokens that share a cache scale (per head)
RUN = 128      # channels in one run of the packed layout


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one action token through the smallest attention projection (hidden 2048): launch
        # latency is what counts
        {"name": "gemv 1x2048x2048 g128", "op": "gemv", "M": 1, "K": 2048, "N": 2048,
         "group": 128, "cinv": False, "bias": True},
        # one token through the fused q/k/v projection of the hidden-4096 block
        {"name": "gemv 1x4096x12288 g128", "op": "gemv", "M": 1, "K": 4096, "N": 12288,
         "group": 128, "cinv": False, "bias": True},
        # eight tokens through its FFN down-projection, with the shared channel scale folded in
        {"name": "gemv 8x16384x4096 g64 cinv", "op": "gemv", "M": 8, "K": 16384, "N": 4096,
         "group": 64, "cinv": True, "bias": True},
        # sixteen action tokens through an odd number of output channels (a head's shard),
        # the finest groups
        {"name": "gemv 16x8192x8191 g32", "op": "gemv", "M": 16, "K": 8192, "N": 8191,
         "group": 32, "cinv": False, "bias": False},
        # packing a small projection, and the largest weight of the hidden-4096 block
        {"name": "pack 2048x2048 g128", "op": "pack", "K": 2048, "N": 2048, "group": 128,
         "c": False},
        {"name": "pack 16384x4096 g64 c", "op": "pack", "K": 4096, "N": 16384, "group": 64,
         "c": True},
        # a decoding step: one new token for each of 32 sequences
        {"name": "append 32x1 h8 d128", "op": "append", "B": 32, "new": 1, "past": 3000,
         "heads": 8, "D": 128, "page": 64},
        # the context of the hidden-4096 block (8512 tokens, 32 heads) written in one call for
        # three sequences of different lengths
        {"name": "append 3x4256 h32 d128", "op": "append", "B": 3, "new": 4256, "past": 37,
         "heads": 32, "D": 128, "page": 64},
        # one token of one short sequence: latency
        {"name": "attn 1x1 kv500 h16/16", "op": "attn", "B": 1, "Lq": 1, "kv": 500, "Hq": 16,
         "Hkv": 16, "D": 128, "page": 16, "causal": True},
        # a decoding step over 32 ragged sequences, four query heads to a cache head
        {"name": "attn 32x1 kv8192 h32/8", "op": "attn", "B": 32, "Lq": 1, "kv": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "causal": True},
        # two long contexts
        {"name": "attn 2x1 kv131072 h32/8", "op": "attn", "B": 2, "Lq": 1, "kv": 131072,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "causal": True},
        # a chunk of up to 64 action tokens that attends to the whole cached context
        # (video, proprio and action tokens) of another length, every head with its own cache
        {"name": "attn 2x64 kv8512 h32/32 full", "op": "attn", "B": 2, "Lq": 64, "kv": 8512,
         "Hq": 32, "Hkv": 32, "D": 64, "page": 32, "causal": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "pack", "append", "attn", "attn", "attn"])
    if op in ("gemv", "pack"):
        K = 128 * _log(rng, 1, 128)
        N = _log(rng, 1, min(16384, 67108864 // K))
        group = rng.choice([32, 64, 128])
        if op == "pack":
            return {"op": op, "K": K, "N": N, "group": group, "c": rng.random() < 0.5}
        return {"op": op, "M": rng.randint(1, 16), "K": K, "N": N, "group": group,
                "cinv": rng.random() < 0.5, "bias": rng.random() < 0.5}
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        new = _log(rng, 1, 4256)
        heads = max(1, min(_log(rng, 1, 32), 400000 // (B * new)))
        new = min(new, 400000 // (B * heads))
        return {"op": op, "B": B, "new": new, "past": _log(rng, 1, 4000) - 1, "heads": heads,
                "D": D, "page": page}
    Hkv, G = _log(rng, 1, 32), rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    Hkv = min(Hkv, max(1, 64 // G))
    Lq = rng.choice([1, 1, _log(rng, 2, 64)])
    B = _log(rng, 1, 64)
    kv = _log(rng, max(1, Lq), min(131072, max(Lq + 1, 1000000 // (B * Hkv * -(-Lq * G // 64)))))
    return {"op": op, "B": B, "Lq": Lq, "kv": kv, "Hq": Hkv * G, "Hkv": Hkv, "D": D,
            "page": page, "causal": rng.random() < 0.7}


def _ragged(count, most, least, salt):
    """Lengths from a tenth of `most` up to it, the first one `most`: of the case alone."""
    r = random.Random(salt * 1000003 + count * 131 + most)
    return [most] + [max(least, r.randint(most // 10, most)) for _ in range(count - 1)]


def _lengths(case):
    if case["op"] == "append":
        return (_ragged(case["B"], case["new"], 1, 1),
                [r for r in _ragged(case["B"], case["past"], 0, 2)])
    Lq = _ragged(case["B"], case["Lq"], 1, 3)
    return Lq, [max(a, b) for a, b in zip(Lq, _ragged(case["B"], case["kv"], 1, 4))]


def work(case):
    if case["op"] in ("gemv", "pack"):
        K, N = case["K"], case["N"]
        packed = N * K / 2 + 2 * N * K / case["group"]
        if case["op"] == "pack":
            return {"bytes": 2 * N * K + packed + (4 * K if case["c"] else 0), "flops": 2 * N * K}
        M = case["M"]
        return {"bytes": packed + 2 * M * (K + N) + (4 * K if case["cinv"] else 0)
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    D = case["D"]
    if case["op"] == "append":
        new, past = _lengths(case)
        T, H = sum(new), case["heads"]
        blocks = sum((p + n - 1) // BLOCK - p // BLOCK + 1 for n, p in zip(new, past))
        return {"bytes": 2 * T * H * D * 3 + 8 * blocks * H + 12 * case["B"], "flops": 4 * T * H * D}
    Lq, kv = _lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    tokens = sum(kv)
    seen = sum(q * n - (q * (q - 1) // 2 if case["causal"] else 0) for q, n in zip(Lq, kv))
    return {"bytes": tokens * Hkv * (2 * D + 8 / BLOCK) + sum(Lq) * Hq * (4 * D + 4)
            + 4 * sum(-(-n // case["page"]) for n in kv), "flops": 4 * D * Hq * seen}


# ---------------------------------------------------------------- inputs

def _weights(case, g):
    """W ~ N(0, 0.02^2), a few input channels larger, as a projection has them."""
    K, N = case["K"], case["N"]
    W = torch.randn(N, K, generator=g, device="cuda") * 0.02
    return W.to(torch.bfloat16)


def _channel_scale(K, g):
    return torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5)


def _tables(lens, page, g):
    """A block table over pages in random order, with a few pages that no sequence has."""
    need = [-(-n // page) for n in lens]
    width, total = max(1, max(need)), sum(need) + 5
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("gemv", "pack"):
        K, N, G = case["K"], case["N"], case["group"]
        s["qw"] = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
        s["s_g"] = torch.zeros(K // G, N, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "pack":
            s["W"] = _weights(case, g)
            s["c_k"] = _channel_scale(K, g) if case["c"] else None
            return s
        M = case["M"]
        # random codes: every layout of bytes is some matrix of codes; -8 does not occur in a
        # packed weight, so its nibble becomes 7's
        q = torch.randint(-7, 8, (N, K), generator=g, device="cuda", dtype=torch.int32)
        s["qw"] = _pack_codes(q)
        s["s_g"] = (torch.rand(K // G, N, generator=g, device="cuda") * 0.006 + 0.004).bfloat16()
        s["x"] = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        s["cinv_k"] = 1 / _channel_scale(K, g) if case["cinv"] else None
        s["b_n"] = torch.randn(N, generator=g, device="cuda") * 0.01 if case["bias"] else None
        s["y"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        return s
    D, P = case["D"], case["page"]
    H = case["heads"] if case["op"] == "append" else case["Hkv"]
    Lq, n = _lengths(case)
    lens = [a + b for a, b in zip(Lq, n)] if case["op"] == "append" else n
    s["table"], pages = _tables(lens, P, g)
    for t in ("k", "v"):
        s[t + "_codes"] = torch.randint(-127, 128, (pages, H, P, D), generator=g, device="cuda",
                                        dtype=torch.int8)
        s[t + "_scale"] = torch.rand(pages, H, P // BLOCK, generator=g,
                                     device="cuda") * 0.012 + 0.018
    s["start"] = _starts(Lq)
    T = sum(Lq)
    if case["op"] == "append":
        s["past_len"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        # keys and values as the fused projection leaves them: parts of wider rows
        qkv = torch.randn(T, 3, H, D, generator=g, device="cuda").bfloat16()
        s["k"], s["v"] = qkv[:, 1], qkv[:, 2]
        return s
    Hq = case["Hq"]
    s["kv_len"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    s["q"] = (torch.randn(T, Hq, D, generator=g, device="cuda") * 1.5).bfloat16()
    s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(T, Hq, device="cuda")
    if own:
        import activation_quantized_gemm_wq_b200 as wq
        s["ws"] = wq.alloc_attn_workspace(T, case["B"], Hq, H, D)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"gemv": _gemv, "pack": _pack, "append": _append, "attn": _attn}[s["op"]](s)


# A run of 128 channels of one row is 64 bytes, sixteen 32-bit words.  Word 4t + j
# (t, j = 0..3) holds channels 32 j + 8 t .. + 7; of these eight, channel 2 i is nibble i and
# channel 2 i + 1 nibble i + 4.

def _pack_codes(q):
    N, K = q.shape
    q = (q & 15).view(N, K // RUN, 4, 4, 4, 2)               # [run][j][t][i][odd]
    word = q.permute(0, 1, 3, 2, 5, 4).reshape(N, K // 8, 8)   # [run][t][j] words of nibbles
    return (word[..., 0::2] | (word[..., 1::2] << 4)).to(torch.uint8).reshape(N, K // 2)


def _unpack_codes(qw):
    N, half = qw.shape
    b = qw.to(torch.int8)
    lo, hi = (b << 4) >> 4, b >> 4                            # sign-extended nibbles
    w = torch.stack([lo, hi], -1).view(N, half // 64, 4, 4, 2, 4)   # [run][t][j][odd][i]
    return w.permute(0, 1, 3, 2, 5, 4).reshape(N, half * 2)


def _gemv(s):
    if own:
        import activation_quantized_gemm_wq_b200 as wq
        wq.wq_gemv_w4g(s["x"], s["cinv_k"], s["qw"], s["s_g"], s["group"], s["b_n"], s["y"])
        return s["y"]
    x = s["x"].float()
    if s["cinv_k"] is not None:
        x = x * s["cinv_k"]
    w = _unpack_codes(s["qw"]).float() * s["s_g"].float().repeat_interleave(s["group"], 0).t()
    y = x @ w.t()
    if s["b_n"] is not None:
        y = y + s["b_n"]
    return y.bfloat16()


def _pack(s):
    # the packed bytes and the scales are the operator's result; the bytes are whole numbers
    if own:
        import activation_quantized_gemm_wq_b200 as wq
        wq.wq_pack_int4_group(s["W"], s["c_k"], s["group"], s["qw"], s["s_g"])
        return {"qw": s["qw"], "s_g": s["s_g"]}
    w = s["W"].float()
    if s["c_k"] is not None:
        w = w * s["c_k"]
    N, K = w.shape
    w = w.view(N, K // s["group"], s["group"])
    # the quotients are rounded to fp32 and to bf16 in this order: a code is decided by them
    # (divided by a tensor: torch multiplies by the reciprocal of a number)
    sc = (w.abs().amax(-1) / w.new_full((), 7.0)).bfloat16()
    q = torch.round(w / sc.float()[..., None]).clamp(-7, 7)
    q = torch.where(sc[..., None] == 0, torch.zeros_like(q), q)
    return {"qw": _pack_codes(q.to(torch.int32).view(N, K)), "s_g": sc.t().contiguous()}


def _rows(start, T):
    """For every packed row its sequence and its place in it."""
    r = torch.arange(T, device=start.device)
    b = torch.searchsorted(start, r.to(torch.int32), right=True) - 1
    return b, r - start[b]


def _append(s):
    # the cache itself is the operator's result: int8 codes, whole numbers, and their scales
    if own:
        import activation_quantized_gemm_wq_b200 as wq
        wq.wq_kv8_append(s["k"], s["v"], s["start"], s["past_len"], s["table"], s["k_codes"],
                         s["v_codes"], s["k_scale"], s["v_scale"])
    else:
        P, T = s["page"], s["k"].shape[0]
        b, i = _rows(s["start"], T)
        pos = s["past_len"][b] + i
        page = s["table"][b, pos // P].long()
        blk = (pos % P) // BLOCK
        # the block in which each sequence goes on: its old codes take the new scale
        first, old = s["past_len"] // BLOCK * BLOCK, s["past_len"] % BLOCK
        seq = torch.arange(len(old), device=old.device)
        opage = s["table"][seq, (first // P).clamp(max=s["table"].shape[1] - 1)].long()
        oblk = (first % P) // BLOCK
        keep = (torch.arange(BLOCK, device=old.device) < old[:, None])[:, None, :, None]
        for t in ("k", "v"):
            x, codes, scale = s[t].float(), s[t + "_codes"], s[t + "_scale"]
            H, D = x.shape[1:]
            blocks = codes.view(-1, H, P // BLOCK, BLOCK, D)
            before = scale[opage, :, oblk]
            fresh = scale.clone()
            fresh[page, :, blk] = 0
            fresh[opage, :, oblk] = torch.where(old[:, None] > 0, before, fresh[opage, :, oblk])
            flat = (page * (P // BLOCK) + blk)[:, None] * H + torch.arange(H, device=x.device)
            by = fresh.permute(0, 2, 1).reshape(-1).scatter_reduce(
                0, flat.reshape(-1), (x.abs().amax(-1) / x.new_full((), 127.0)).reshape(-1),
                "amax")
            scale.copy_(by.view(-1, P // BLOCK, H).permute(0, 2, 1))
            now = scale[opage, :, oblk]
            ratio = torch.where(now > 0, before / now, torch.ones_like(now))[..., None, None]
            was = blocks[opage, :, oblk]
            again = torch.round(was.float() * ratio).to(torch.int8)
            blocks[opage, :, oblk] = torch.where(keep & (now > before)[..., None, None], again, was)
            sc = scale[page, :, blk][..., None]
            q = torch.round(x / sc).clamp(-127, 127)
            codes[page, :, pos % P] = torch.where(sc == 0, torch.zeros_like(q), q).to(torch.int8)
    return {n: s[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale")}


def _attn(s):
    D = s["D"]
    if own:
        import activation_quantized_gemm_wq_b200 as wq
        wq.wq_attn_kv8(s["q"], s["start"], s["kv_len"], s["table"], s["k_codes"], s["v_codes"],
                       s["k_scale"], s["v_scale"], s["causal"], D ** -0.5, s["out"], s["lse"],
                       s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Lq, Hq, Hkv = s["B"], s["Lq"], s["Hq"], s["Hkv"]
    G, n = Hq // Hkv, s["table"].shape[1] * s["page"]

    def whole(codes, scale):      # [B][Hkv][n][D] in fp32
        t = s["table"].long()
        c = codes[t].float().view(B, -1, Hkv, s["page"] // BLOCK, BLOCK, D)
        c = c * scale[t][..., None, None]
        return c.permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, n, D)

    b, i = _rows(s["start"], s["q"].shape[0])
    q = torch.zeros(B, Lq, Hq, D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, Lq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Lq * G, D)
    p = (q @ whole(s["k_codes"], s["k_scale"]).transpose(2, 3)) * D ** -0.5
    p = p.view(B, Hkv, Lq, G, n)
    lens = s["kv_len"].view(B, 1, 1, 1, 1)
    col = torch.arange(n, device="cuda")
    see = col < lens
    if s["causal"]:
        nq = (s["start"][1:] - s["start"][:-1]).view(B, 1, 1, 1, 1)
        at = torch.arange(Lq, device="cuda").view(1, 1, Lq, 1, 1)
        see = see & (col <= lens - nq + at)
    p = p.masked_fill(~see, -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(p - top)
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, Lq * G, n) @ whole(s["v_codes"], s["v_scale"])
    o = o.view(B, Hkv, Lq, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Lq, Hq, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, Lq, Hq)
    return {"out": o[b, i].bfloat16(), "lse": lse[b, i].contiguous()}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "pack":
        w = s["W"].to(f8)
        if s["c_k"] is not None:
            w *= s["c_k"].to(f8)
        parts = [w[:, k:k + case["group"]].abs().max(1).values / 7
                 for k in range(0, case["K"], case["group"])]
        return {"qw": None, "s_g": torch.stack(parts)}
    if case["op"] == "gemv":
        words = s["qw"].cpu().view(torch.int32).view(case["N"], case["K"] // RUN, 16).cuda()
        w = torch.empty(case["N"], case["K"], dtype=f8, device="cuda")
        by_run = w.view(case["N"], case["K"] // RUN, RUN)
        for at in range(16):
            t, j = at // 4, at % 4
            for e in range(8):
                nib = (words[:, :, at] >> (4 * (e // 2 + 4 * (e % 2)))) & 15
                by_run[:, :, 32 * j + 8 * t + e] = (nib - 16 * (nib > 7).int()).to(f8)
        for j in range(case["K"] // case["group"]):
            w[:, j * case["group"]:(j + 1) * case["group"]] *= s["s_g"][j].to(f8)[:, None]
        x = s["x"].to(f8)
        if s["cinv_k"] is not None:
            x = x * s["cinv_k"].to(f8)
        y = torch.einsum("mk,nk->mn", x, w)
        return y if s["b_n"] is None else y + s["b_n"].to(f8)
    if case["op"] == "append":
        new, past = _lengths(case)
        if case["B"] * max(new) > 40000 and case["B"] > 8:
            return None
        out = {"k_codes": None, "v_codes": None}
        table, start = s["table"].tolist(), s["start"].tolist()
        for t in ("k", "v"):
            scale = s[t + "_scale"].to(f8)
            for b in range(case["B"]):
                p, end = past[b], past[b] + new[b]
                while p < end:
                    stop = min(end, p // BLOCK * BLOCK + BLOCK)
                    at = start[b] + p - past[b]
                    a = s[t][at:at + stop - p].to(f8).abs().amax((0, 2)) / 127
                    to = scale[table[b][p // case["page"]], :, p % case["page"] // BLOCK]
                    to.copy_(torch.maximum(a, to) if p % BLOCK else a)
                    p = stop
            out[t + "_scale"] = scale
        return out
    Lq, kv = _lengths(case)
    D, G, P = case["D"], case["Hq"] // case["Hkv"], case["page"]
    out = torch.empty(sum(Lq), case["Hq"], D, dtype=f8, device="cuda")
    lse = torch.empty(sum(Lq), case["Hq"], dtype=f8, device="cuda")
    at = 0
    for b, (m, n) in enumerate(zip(Lq, kv)):
        pages = s["table"][b, :-(-n // P)].long()
        for h in range(case["Hkv"]):
            k, v = (torch.repeat_interleave(s[t + "_scale"][pages, h].to(f8).flatten(), BLOCK)[:n]
                    [:, None] * s[t + "_codes"][pages, h].reshape(-1, D)[:n].to(f8)
                    for t in ("k", "v"))
            for j in range(h * G, h * G + G):
                x = s["q"][at:at + m, j].to(f8) @ k.T / math.sqrt(D)
                if case["causal"]:
                    hidden = torch.arange(n, device="cuda")[None] > \
                        n - m + torch.arange(m, device="cuda")[:, None]
                    x[hidden] = -math.inf
                lse[at:at + m, j] = torch.logsumexp(x, 1)
                out[at:at + m, j] = torch.softmax(x, 1) @ v
        at += m
    return {"out": out, "lse": lse}

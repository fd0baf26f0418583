"""The group-scaled product where its value is decided by few bits: tokens and weights whose
terms cancel, and values at the ends of the range.  Against 64-bit sums."""
import pytest
import torch

from test_gpu_group import codes_of, gemv, packed

pytestmark = pytest.mark.gpu


def in_64_bits(x, cinv, qw, s_g, group):
    """(y, sum of the terms' magnitudes, x', weights)."""
    x8 = x.double() if cinv is None else x.double() * cinv.double()
    w = torch.from_numpy(codes_of(qw.cpu().numpy())).cuda().double()
    w = w * s_g.double().t().repeat_interleave(group, 1)
    return x8 @ w.t(), x8.abs() @ w.abs().t(), x8, w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K", [(1, 512), (3, 512), (5, 512), (8, 2048), (9, 512), (16, 1024),
                                 (12, 32768)])
def test_scaled_tokens_keep_their_bits(M, K, group):
    """Neighbouring channels with equal weights, opposite tokens and channel scales that
    differ by 2^-13: what is left of their terms is in the low bits of x * cinv, which 11
    bits do not have.  Allowed: half a bf16 step; x' off by 2^-22 of its group's largest (that
    covers 2^-22 of itself); a group's sum in at most 16 matrix steps, each within 2^-22 of
    the terms' magnitudes; the fp32 product of x and cinv, four operations to a group's term and
    the additions over groups and parts, each 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(M * K + group)
    N = 37
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.02).bfloat16()
    W[:, 1::2] = W[:, 0::2]
    qw, s_g = packed(W, None, group)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    x[:, 1::2] = -x[:, 0::2]
    cinv = torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5)
    cinv[1::2] = cinv[0::2] * (1 + 2.0 ** -13 * torch.rand(K // 2, generator=g, device="cuda"))
    y = gemv(x, cinv, qw, s_g, group, None)
    want, size, x8, w = in_64_bits(x, cinv, qw, s_g, group)
    top = x8.abs().view(M, K // group, group).amax(-1).repeat_interleave(group, 1)
    allow = want.abs() * 2.0 ** -8 + (top * 2.0 ** -22) @ w.abs().t() \
        + size * ((K / group + 8 + 5) * 2.0 ** -24 + 16 * 2.0 ** -22) + 2.0 ** -133
    off = (y.double() - want).abs()
    assert bool((off <= allow).all()), float((off / allow).max())


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("M", [1, 3, 5, 8, 9, 16])
@pytest.mark.parametrize("size,weight", [(3e38, 2.0 ** -20), (3e38, 2.0 ** -100), (2.0 ** -60, 2.0 ** 100),
                                         (2.0 ** -110, 2.0 ** 20), (2.0 ** -115, 0.25)])
def test_tokens_and_scales_at_the_ends_of_the_range(size, weight, M, scaled, group):
    """Tokens up to bf16's largest against small weight scales, and the other way round, with the
    code -8, which packing never makes but a byte can hold: y is in range, and so is every sum
    on the way.  Allowed as above, and at bf16's lower end 2^-133: half of its smallest step
    and as much for the sums' own."""
    K, N = 512, 24
    g = torch.Generator(device="cuda").manual_seed(M + group)
    qw = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    qw[:2] = 0x88                                          # -8 everywhere: the largest sums
    s_g = ((torch.rand(K // group, N, generator=g, device="cuda") + 0.5) * weight).bfloat16()
    x = (torch.rand(M, K, generator=g, device="cuda") * 0.75 + 0.25) * size
    x = (x * torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.3, -1.0, 1.0)).bfloat16()
    cinv = torch.rand(K, generator=g, device="cuda") * 0.5 + 0.5 if scaled else None
    y = gemv(x, cinv, qw, s_g, group, None)
    want, sizes, x8, w = in_64_bits(x, cinv, qw, s_g, group)
    top = x8.abs().view(M, K // group, group).amax(-1).repeat_interleave(group, 1)
    allow = want.abs() * 2.0 ** -8 + (top * 2.0 ** -22 + 2.0 ** -128) @ w.abs().t() \
        + sizes * ((K / group + 8 + 5) * 2.0 ** -24 + 16 * 2.0 ** -22) + 2.0 ** -133
    off = (y.double() - want).abs()
    assert bool((off <= allow).all()), float((off / allow).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_a_weight_that_is_not_finite_is_seen(bad, group):
    """One weight is not finite, or its product with the channel scale is not: its group's scale
    says so, and so does every product of its row; all else is what it is without it."""
    N, K, n, k = 21, 512, 13, 300
    g = torch.Generator(device="cuda").manual_seed(group)
    W = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    c = torch.full((K,), 4.0, device="cuda")
    calm = packed(W, c, group)
    W[n, k] = bad
    qw, s_g = packed(W, c, group)
    assert not bool(s_g[k // group, n].isfinite())
    for M in (1, 3, 8, 16):
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        x[0] = 0
        y, want = gemv(x, None, qw, s_g, group, None), gemv(x, None, *calm, group, None)
        assert not bool(y[:, n].isfinite().any())
        y[:, n] = want[:, n]
        assert torch.equal(y, want)
    run = slice(k // 128 * 64, k // 128 * 64 + 64)
    qw[n, run], s_g[k // group, n] = calm[0][n, run], calm[1][k // group, n]
    assert torch.equal(qw, calm[0]) and torch.equal(s_g, calm[1])

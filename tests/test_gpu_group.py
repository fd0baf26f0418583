"""int4 weights with a scale per group of channels: the packing bit for bit against
numpy, the product of 1 to 16 tokens against 64-bit sums."""
import numpy as np
import pytest
import torch

import activation_quantized_gemm_wq_b200 as wq

pytestmark = pytest.mark.gpu


def codes_of(qw):
    """The packed layout as include/wq.h words it: word 4t + j of a 64-byte run holds
    channels 32j + 8t .. + 7, channel 2i in nibble i and 2i + 1 in nibble i + 4."""
    qw = np.ascontiguousarray(qw)
    N, half = qw.shape
    words = qw.view("<u4").reshape(N, half // 64, 16)
    q = np.empty((N, half // 64, 128), np.int64)
    for t in range(4):
        for j in range(4):
            for c in range(8):
                nib = (words[:, :, 4 * t + j] >> (4 * (c // 2 + 4 * (c % 2)))) & 15
                q[:, :, 32 * j + 8 * t + c] = nib.astype(np.int64) - 16 * (nib >= 8)
    return q.reshape(N, half * 2)


def packed(W, c, group):
    N, K = W.shape
    qw = torch.full((N, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    s_g = torch.full((K // group, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    wq.wq_pack_int4_group(W.cuda(), None if c is None else c.cuda(), group, qw, s_g)
    return qw, s_g


def pack_reference(W, c, group):
    """(codes, scales) in IEEE fp32, the scale rounded to bf16 before the codes."""
    w = W.float().numpy()
    if c is not None:
        w = w * c.numpy()[None, :]
    N, K = w.shape
    w = w.reshape(N, K // group, group)
    s = torch.from_numpy(np.abs(w).max(-1) / np.float32(7)).bfloat16()
    sf = s.float().numpy()[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(sf == 0, np.float32(0), np.clip(np.rint(w / sf), -7, 7))
    return q.reshape(N, K).astype(np.int64), s.t().contiguous()


@pytest.mark.parametrize("N,K,group,scaled", [
    (1, 128, 32, False), (1, 128, 128, True), (17, 384, 64, True), (33, 1024, 32, True),
    (128, 2048, 128, False), (5, 32768, 64, True)])
def test_pack_is_bit_exact(N, K, group, scaled):
    g = torch.Generator().manual_seed(N * K + group)
    W = (torch.randn(N, K, generator=g) * 0.02).bfloat16()
    W[0, :group] = 0                                   # an empty group: scale 0, codes 0
    # multiples of half a step around the group's maximum: ties of the rounding
    W[-1, -group:] = (torch.arange(group) % 15 - 7).bfloat16() / 2
    W[-1, -1] = 7
    c = torch.exp(torch.randn(K, generator=g)) if scaled else None
    qw, s_g = packed(W, c, group)
    q, s = pack_reference(W, c, group)
    assert torch.equal(s_g.cpu().view(torch.int16), s.view(torch.int16))
    assert np.array_equal(codes_of(qw.cpu().numpy()), q)


@pytest.mark.parametrize("size", [1e-38, 3e-39, 1e36])
def test_pack_at_the_ends_of_the_range(size):
    """Scales that are subnormal, whose reciprocal overflows, and huge ones."""
    g = torch.Generator().manual_seed(3)
    W = (torch.randn(16, 256, generator=g) * size).bfloat16()
    qw, s_g = packed(W, None, 64)
    q, s = pack_reference(W, None, 64)
    assert torch.equal(s_g.cpu().view(torch.int16), s.view(torch.int16))
    assert np.array_equal(codes_of(qw.cpu().numpy()), q)


def gemv(x, cinv, qw, s_g, group, bias):
    y = torch.full((x.shape[0], qw.shape[0]), float("nan"), dtype=torch.bfloat16, device="cuda")
    wq.wq_gemv_w4g(x, cinv, qw, s_g, group, bias, y)
    return y


def check_gemv(x, cinv, qw, s_g, group, bias, y):
    """y against 64-bit sums.  One rounding to bf16 (half a step: 2^-8 relative, and the
    subnormals' 2^-134); fp32 sums over the K / group groups and at most 8 parts, with four
    operations to a group's term, each within 2^-24 of the sum of magnitudes; and, up to
    four tokens, x' held to 2^-22 of its group's largest (or 2^-128), summed exactly; beyond
    four, x' in f16 (2^-11 relative, exact for bf16 itself; 2^-39 of the group's largest
    where that is subnormal) and at most 8 matrix steps to a group's sum, each within 2^-22."""
    x8 = x.double()
    if cinv is not None:
        x8 = x8 * cinv.double()
    w = torch.from_numpy(codes_of(qw.cpu().numpy())).cuda().double()
    w = w * s_g.double().t().repeat_interleave(group, 1)
    ref = x8 @ w.t()
    size = x8.abs() @ w.abs().t()
    if bias is not None:
        ref, size = ref + bias.double(), size + bias.double().abs()
    K = x.shape[1]
    top = x8.abs().view(-1, K // group, group).amax(-1).repeat_interleave(group, 1)
    few = x.shape[0] <= 4
    held = (top * 2.0 ** (-22 if few else -39) + 2.0 ** -128) @ w.abs().t()
    steps = (K / group + 8 + 4) * 2.0 ** -24
    if not few:
        steps += 8 * 2.0 ** -22 + (2.0 ** -11 if cinv is not None else 0)
    allow = ref.abs() * 2.0 ** -8 + size * steps + held + 2.0 ** -133
    bad = ~((y.double() - ref).abs() <= allow)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs outside the bound"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fold", [False, True])
@pytest.mark.parametrize("M,K,N", [
    (1, 128, 1), (1, 2048, 2048), (2, 384, 15), (3, 1152, 33), (7, 4096, 65), (8, 1024, 257),
    (9, 256, 16), (13, 8192, 47), (16, 2048, 31), (4, 16384, 129), (1, 32768, 3),
    # several tiles to a CTA; K split over clusters; more staged tokens than a CTA holds
    (2, 256, 40000), (6, 16384, 700), (5, 32768, 40), (16, 32768, 50), (12, 28672, 20),
    (11, 1152, 5000)])
def test_gemv(M, K, N, group, fold):
    g = torch.Generator(device="cuda").manual_seed(M * 7919 + K + N)
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.02).bfloat16()
    c = torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5) if fold else None
    qw, s_g = packed(W, c, group)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    x[:, ::97] *= 40                                        # outlier channels
    bias = torch.randn(N, generator=g, device="cuda") if (M + N) % 2 else None
    cinv = None if c is None else 1 / c
    y = gemv(x, cinv, qw, s_g, group, bias)
    check_gemv(x, cinv, qw, s_g, group, bias, y)


def test_gemv_one_hot_tokens_read_back_every_weight():
    """x = e_k: y is the weight itself, rounded to bf16, for every channel and row."""
    K, N, group = 256, 19, 32
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(2)).bfloat16()
    qw, s_g = packed(W, None, group)
    w = torch.from_numpy(codes_of(qw.cpu().numpy())).float() * \
        s_g.cpu().float().t().repeat_interleave(group, 1)
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    for k in range(0, K, 16):
        y = gemv(eye[k:k + 16], None, qw, s_g, group, None)
        assert torch.equal(y.cpu(), w[:, k:k + 16].t().bfloat16())


def test_gemv_of_extreme_values():
    """bf16's whole range passes through: x near the largest and smallest values (the
    products stay finite), and minus eight, which packing never makes but a byte can hold."""
    g = torch.Generator(device="cuda").manual_seed(8)
    N, K, group = 40, 512, 64
    qw = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s_g = torch.rand(K // group, N, generator=g, device="cuda").bfloat16() * 1e-4
    x = torch.randn(3, K, generator=g, device="cuda")
    x[1] *= 1e34
    x[2] *= 1e-34
    x = x.bfloat16()
    check_gemv(x, None, qw, s_g, group, None, gemv(x, None, qw, s_g, group, None))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16])
def test_gemv_of_products_beyond_the_range_is_not_finite(M, group):
    """x and cinv are finite, x * cinv is not: every y of that token says so, and the other
    tokens have what they have without it."""
    K, N = 512, 48
    g = torch.Generator().manual_seed(M)
    qw, s_g = packed(torch.randn(N, K, generator=g).bfloat16(), None, group)
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    cinv = torch.ones(K, device="cuda")
    cinv[77] = 16.0
    calm = gemv(x, cinv, qw, s_g, group, None)
    x[M // 2, 77] = 3e38
    y = gemv(x, cinv, qw, s_g, group, None)
    assert not bool(torch.isfinite(y[M // 2]).any())
    others = [m for m in range(M) if m != M // 2]
    assert torch.equal(y[others], calm[others])


def test_gemv_leaves_what_it_does_not_own():
    """Nothing is written behind y, whatever its alignment, and nothing is read behind qw."""
    K, N, group = 256, 21, 64
    W = (torch.randn(N, K) * 0.02).bfloat16()
    qw, s_g = packed(W, None, group)
    x = torch.randn(5, K, device="cuda").bfloat16()
    room = torch.full((5 * N + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = room[1:1 + 5 * N].view(5, N)                        # 2-byte aligned
    wq.wq_gemv_w4g(x, None, qw, s_g, group, None, y)
    check_gemv(x, None, qw, s_g, group, None, y)
    assert room[0] == 7 and bool((room[1 + 5 * N:] == 7).all())


def test_gemv_empty_batch_and_streams():
    K, N, group = 1024, 64, 128
    W = (torch.randn(N, K) * 0.02).bfloat16()
    qw, s_g = packed(W, None, group)
    wq.wq_gemv_w4g(torch.empty(0, K, dtype=torch.bfloat16, device="cuda"), None, qw, s_g, group,
                   None, torch.empty(0, N, dtype=torch.bfloat16, device="cuda"))
    x = torch.randn(4, K, device="cuda").bfloat16()
    y = [torch.zeros(4, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    wq.wq_gemv_w4g(x, None, qw, s_g, group, None, y[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    wq.wq_gemv_w4g(x, None, qw, s_g, group, None, y[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.wq_gemv_w4g(x, None, qw, s_g, group, None, y[2])
    y[2].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    x.mul_(-1)                                              # the replay reads x as it is then
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[2], -y[0])
    assert wq.wq_device_status() == ("WQ_OK", 0)

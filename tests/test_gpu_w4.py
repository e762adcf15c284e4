"""The 4-bit linear and its converters on the GPU against 64 bits."""
from __future__ import annotations

import pytest

from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def codes_scales(N, K, G, seed, low=-8):
    g = gen(seed)
    codes = torch.randint(low, 8, (N, K), generator=g, device="cuda",
                          dtype=torch.int8)
    scales = torch.exp(torch.randn(N, K // G, generator=g, device="cuda") * 0.3
                       - 4).to(BF)
    return codes, scales


def weight(codes, scales):
    """The weight in 64 bits."""
    N, K = codes.shape
    G = K // scales.shape[1]
    return (codes.double().view(N, -1, G) * scales.double()[:, :, None]).view(
        N, K)


def unpacked(w4, w4_scale):
    """(codes [N, K], scales [N, K/G]) of a packed weight, read by the
    layout's definition one index at a time."""
    nb, kb = w4.shape[:2]
    N, K, G = 16 * nb, 128 * kb, 128 // w4_scale.shape[3]
    n = torch.arange(N)[:, None]
    k = torch.arange(K)[None, :]
    byte = w4.cpu()[n // 16, k // 128, 16 * (k % 32 // 8) + n % 16,
                    4 * (k % 128 // 32) + k % 4].int()
    codes = torch.where(k % 8 < 4, byte % 16, byte // 16) - 8
    g = torch.arange(K // G)[None, :]
    scales = w4_scale.cpu()[n // 16, g * G // 128, n % 16, g * G % 128 // G]
    return codes, scales


SHAPES = [(16, 128), (16, 384), (48, 256), (112, 1152), (272, 128),
          (1024, 640)]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K", SHAPES)
def test_pack_weight(N, K, G):
    say(f"w4 pack {N}x{K} G={G}")
    codes, scales = codes_scales(N, K, G, N + K)
    codes.view(-1)[:6] = torch.tensor([-128, -9, 8, 127, 7, -8],
                                      dtype=torch.int8)
    w4, s = B.w4_pack_weight(codes, scales)
    c2, s2 = unpacked(w4, s)
    assert torch.equal(c2, codes.cpu().int().clamp(-8, 7))
    assert torch.equal(s2.view(torch.int16), scales.cpu().view(torch.int16))


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K", SHAPES)
def test_quantize_weight(N, K, G):
    """Scale and codes are single binary32 divisions and roundings: equal to
    the same steps on the CPU."""
    say(f"w4 quantize {N}x{K} G={G}")
    g = gen(N * 7 + K)
    w = (0.05 * torch.randn(N, K, generator=g, device="cuda")).to(BF)
    w[0, :G] = 0
    w[1, :G] = 2.0 ** -133 * (torch.arange(G, device="cuda") % 4 - 1)
    w[2, :G] = 3.0e38 * (torch.arange(G, device="cuda") % 2 * 2 - 1)
    w[3, :G] = torch.linspace(-7, 7, G, device="cuda").to(BF)
    w4, s = B.w4_quantize_weight(w, group=G)
    codes, scales = unpacked(w4, s)
    f = w.float().cpu().view(N, K // G, G)
    amax = f.abs().amax(2)
    want = (amax / 7).to(BF)
    want = torch.where(want == 0, torch.tensor(2.0 ** -133, dtype=BF), want)
    want = torch.where(amax == 0, torch.tensor(1.0, dtype=BF), want)
    assert torch.equal(scales.view(torch.int16), want.view(torch.int16))
    q = torch.round(f / want.float()[:, :, None]).clamp(-7, 7).int()
    assert torch.equal(codes, q.view(N, K))


def check(x, codes, scales, bias, y):
    """Each product and sum in binary32 in any order: G + K / 128 + 16
    roundings at most lie on an input's way to its output, counted double for
    the matrix instruction's own rounding, over magnitudes of |x| (|code| + 16)
    s (the -8 and the offset code are added apart)."""
    N, K = codes.shape
    G = K // scales.shape[1]
    xd, w = x.double(), weight(codes, scales)
    want = xd @ w.t().contiguous()
    mag = xd.abs() @ weight(codes.abs() + 16, scales).t().contiguous()
    if bias is not None:
        want = want + bias.double()
        mag = mag + bias.double().abs()
    e = 2 * (G + K / 128 + 16) * U * mag
    off = (y.double() - want).abs()
    most = e + 2.0 ** -8 * (want.abs() + e) + 2.0 ** -133
    assert (off <= most).all(), (off / most).max()


TOKENS = [1, 2, 3, 7, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 130]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", TOKENS)
def test_linear_exact(M, G):
    """Integer inputs and scales that are powers of two: every sum is exact,
    so the result is the exact one rounded once, bit for bit."""
    say(f"w4 exact M={M} G={G}")
    for N, K in [(16, 128), (48, 384), (272, 2176), (1024, 5376)]:
        g = gen(M * N + G)
        codes, _ = codes_scales(N, K, G, M + N)
        scales = torch.exp2(torch.randint(-3, 2, (N, K // G), generator=g,
                                          device="cuda").float()).to(BF)
        x = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(BF)
        bias = torch.randint(-64, 65, (N,), generator=g, device="cuda").to(BF)
        w4, s = B.w4_pack_weight(codes, scales)
        y = B.w4_linear(x, w4, s, bias)
        want = x.double() @ weight(codes, scales).t().contiguous()
        assert torch.equal(y, (want + bias.double()).float().to(BF)), (N, K)
        y = B.w4_linear(x, w4, s)
        assert torch.equal(y, want.float().to(BF)), (N, K)


@pytest.mark.parametrize("M", [1, 4, 5, 8, 9, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("tiles", [128, 130, 255, 257, 384, 386, 511, 515, 767,
                                   770, 1021, 1027, 1533, 1543, 1800])
def test_linear_exact_wide(M, tiles):
    """Every number of channel tiles a work group takes, the last group with
    fewer; K of fewer blocks than waves and of one more round."""
    say(f"w4 wide M={M} tiles={tiles}")
    for K, G in ((128, 32), (2176, 128)):
        N = 16 * tiles
        g = gen(M * tiles + K)
        codes, _ = codes_scales(N, K, G, M + N)
        scales = torch.exp2(torch.randint(-3, 2, (N, K // G), generator=g,
                                          device="cuda").float()).to(BF)
        x = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(BF)
        w4, s = B.w4_pack_weight(codes, scales)
        raw = torch.full((M * N * 2 + 8192,), 0xA5, dtype=torch.uint8,
                         device="cuda")
        bias = torch.randint(-64, 65, (N,), generator=g, device="cuda").to(BF)
        y = B.w4_linear(x, w4, s, out=raw[4096:-4096].view(BF).view(M, N))
        want = x.double() @ weight(codes, scales).t().contiguous()
        assert torch.equal(y, want.float().to(BF))
        assert torch.equal(B.w4_linear(x, w4, s, bias),
                           (want + bias.double()).float().to(BF))
        assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()


def test_linear_tiny_inputs():
    """Inputs below the normal range of BF16, raised by the scales: products
    and the offset's sum keep them."""
    N, K = 32, 256
    codes, scales = codes_scales(N, K, 128, 5)
    scales[:] = 2.0 ** 100
    x = (torch.randint(-3, 4, (19, K), generator=gen(2), device="cuda").double()
         * 2.0 ** -132).to(BF)
    w4, s = B.w4_pack_weight(codes, scales)
    for M in (3, 19):
        want = x[:M].double() @ weight(codes, scales).t().contiguous()
        assert torch.equal(B.w4_linear(x[:M].contiguous(), w4, s),
                           want.float().to(BF))


def test_linear_every_weight():
    """One-hot tokens read every weight of the layout on its own."""
    N, K = 80, 256
    for G in (32, 64, 128):
        codes, scales = codes_scales(N, K, G, G)
        w4, s = B.w4_pack_weight(codes, scales)
        y = B.w4_linear(torch.eye(K, device="cuda", dtype=BF), w4, s)
        want = weight(codes, scales).t().float().to(BF)
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K,G", [
    (1, 5376, 5376, 128), (5, 5376, 5376, 32), (16, 1000 * 16, 896, 64),
    (17, 16, 21504, 128), (32, 7168, 5376, 64), (64, 5376, 21504, 32),
    (64, 28672, 640, 128), (61, 5392, 1152, 128), (200, 528, 5376, 64)])
def test_linear(M, N, K, G):
    say(f"w4 linear {M}x{N}x{K} G={G}")
    codes, scales = codes_scales(N, K, G, M + N + K)
    g = gen(K)
    x = torch.randn(M, K, generator=g, device="cuda")
    x = torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.001,
                    20 * x, x).to(BF)
    bias = torch.randn(N, generator=g, device="cuda").to(BF)
    w4, s = B.w4_pack_weight(codes, scales)
    raw = torch.full((M * N * 2 + 8192,), 0xA5, dtype=torch.uint8,
                     device="cuda")
    y = raw[4096:-4096].view(BF).view(M, N)
    B.w4_linear(x, w4, s, bias, out=y)
    torch.cuda.synchronize()
    assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()
    check(x, codes, scales, bias, y)
    first = y.clone()
    assert torch.equal(B.w4_linear(x, w4, s, bias), first)  # repeatable


@pytest.mark.parametrize("shift", [1.0, 100.0])
def test_linear_far_from_zero_mean(shift):
    """Inputs all of one sign: the offset's sum is large beside the result."""
    codes, scales = codes_scales(512, 5376, 128, 1)
    x = (shift + 0.1 * torch.randn(9, 5376, generator=gen(2),
                                   device="cuda")).to(BF)
    w4, s = B.w4_pack_weight(codes, scales)
    check(x, codes, scales, None, B.w4_linear(x, w4, s))


def test_quantized_weight_end_to_end():
    """A BF16 weight through the converter: within half a step a weight."""
    N, K, G = 256, 1024, 64
    w = (0.05 * torch.randn(N, K, generator=gen(5), device="cuda")).to(BF)
    w4, s = B.w4_quantize_weight(w, group=G)
    y = B.w4_linear(torch.eye(K, device="cuda", dtype=BF), w4, s).t()
    step = (w.double().view(N, -1, G).abs().amax(2) / 7).repeat_interleave(G, 1)
    # half a step, the rounded scale's 2^-8 of up to 7 steps, the result's
    assert ((y.double() - w.double()).abs() <=
            step * (0.5 + 7 * 2.0 ** -8) + 2.0 ** -8 * w.double().abs() * 1.1
            ).all()


def test_unaligned_bias_and_extreme_scales():
    N, K, G = 64, 256, 32
    codes, scales = codes_scales(N, K, G, 3)
    scales[0] = 2.0 ** -120
    scales[1] = 2.0 ** 100
    scales[2] = 0.0
    scales[3] = -scales[3]
    x = torch.randn(4, K, generator=gen(4), device="cuda").to(BF)
    bias = torch.randn(N + 3, generator=gen(6), device="cuda").to(BF)[3:]
    w4, s = B.w4_pack_weight(codes, scales)
    y = B.w4_linear(x, w4, s, bias)
    xd = x.double() @ weight(codes, scales).t().contiguous() + bias.double()
    mag = (x.double().abs() @ weight(codes.abs() + 16, scales.abs()).t()
           .contiguous() + bias.double().abs())
    e = 2 * (G + K / 128 + 16) * U * mag
    assert ((y.double() - xd).abs() <= e + 2.0 ** -8 * (xd.abs() + e)).all()


def test_nan_stays_in_its_token():
    N, K = 32, 256
    codes, scales = codes_scales(N, K, 64, 3)
    x = torch.randn(20, K, generator=gen(4), device="cuda").to(BF)
    w4, s = B.w4_pack_weight(codes, scales)
    want = B.w4_linear(x, w4, s)
    x[3, 200] = float("nan")
    x[19, 0] = float("inf")
    y = B.w4_linear(x, w4, s)
    rest = [i for i in range(20) if i not in (3, 19)]
    assert torch.equal(y[rest], want[rest])
    assert y[3].isnan().all() and not y[19].isfinite().any()


def test_token_alone_equals_token_in_batch():
    """Tokens are independent: the same bits for any batch of one launch
    path (up to 16 tokens, up to 64)."""
    codes, scales = codes_scales(256, 5376, 128, 8)
    w4, s = B.w4_pack_weight(codes, scales)
    x = torch.randn(130, 5376, generator=gen(9), device="cuda").to(BF)
    small = B.w4_linear(x[:16].contiguous(), w4, s)
    for m in (0, 7, 15):
        assert torch.equal(B.w4_linear(x[m:m + 1].contiguous(), w4, s)[0],
                           small[m])
    big = B.w4_linear(x, w4, s)
    assert torch.equal(B.w4_linear(x[64:128].contiguous(), w4, s), big[64:128])


def test_other_stream_and_graph():
    codes, scales = codes_scales(512, 1280, 64, 8)
    w4, s = B.w4_pack_weight(codes, scales)
    x = torch.randn(24, 1280, generator=gen(9), device="cuda").to(BF)
    want = B.w4_linear(x, w4, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = B.w4_linear(x, w4, s, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    B.w4_linear(x, w4, s, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.w4_linear(x, w4, s, out=y)
    for i in range(3):
        x.copy_(torch.randn(24, 1280, generator=gen(20 + i), device="cuda"))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, B.w4_linear(x, w4, s))


def test_offsets_past_32_bits():
    """A packed weight of more than 2^32 bytes: its last channels."""
    N, K, G = 65616, 130944, 128
    say(f"w4 {N}x{K}")
    w4 = torch.randint(0, 256, (N // 16, K // 128, 64, 16), device="cuda",
                       dtype=torch.uint8, generator=gen(0))
    assert w4.numel() > 2 ** 32
    s = torch.full((N // 16, K // 128, 16, 1), 2.0 ** -6, dtype=BF,
                   device="cuda")
    x = torch.randint(-3, 4, (3, K), device="cuda", generator=gen(1)).to(BF)
    y = B.w4_linear(x, w4, s)
    for t in (0, N // 32, N // 16 - 1):
        codes, scales = unpacked(w4[t:t + 1], s[t:t + 1])
        want = x.double().cpu() @ (codes.double() * 2.0 ** -6).t()
        assert torch.equal(y[:, 16 * t:16 * t + 16].cpu(),
                           want.float().to(BF))

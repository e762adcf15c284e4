"""Channels of zeros and inputs near the ends of BF16's range, through the 4-bit
linear."""
from __future__ import annotations

import pytest

from tests.test_gpu_w4 import check, codes_scales, gen, say
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
TOKENS = [1, 4, 5, 9, 16, 17, 40, 64]


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", TOKENS)
def test_zero_weights(M, G):
    """Channels of zeros (scale 1, every code 8) give the bias, within the
    roundings that the offset costs."""
    say(f"w4 zero weights M={M} G={G}")
    N, K = 272, 1152
    codes, scales = codes_scales(N, K, G, M + G)
    codes[::3] = 0
    scales[::3] = 1.0
    x = (100 + torch.randn(M, K, generator=gen(G), device="cuda")).to(BF)
    bias = torch.randn(N, generator=gen(M), device="cuda").to(BF)
    w4, s = B.w4_pack_weight(codes, scales)
    check(x, codes, scales, bias, B.w4_linear(x, w4, s, bias))
    # whole numbers leave no rounding behind
    x = torch.randint(-255, 256, (M, K), generator=gen(M), device="cuda").to(BF)
    y = B.w4_linear(x, w4, s, bias)
    assert torch.equal(y[:, ::3], bias[::3].expand(M, -1))


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", TOKENS)
def test_inputs_near_the_end_of_the_range(M, G):
    """Inputs of 2^127 and nearly 2^127 the other way in every group, under any
    code: the sums stay finite, as the result does."""
    say(f"w4 near the end M={M} G={G}")
    N, K = 112, 640
    codes, scales = codes_scales(N, K, G, M + 1)
    scales = (scales.float() * 2.0 ** -10).to(BF)
    codes[::5, 7::G] = 0
    codes[::7, 21::G] = -8
    x = torch.randn(M, K, generator=gen(M), device="cuda").to(BF)
    x[:, 7::G] = 2.0 ** 127
    x[:, 21::G] = -1.9921875 * 2.0 ** 126
    w4, s = B.w4_pack_weight(codes, scales)
    y = B.w4_linear(x, w4, s)
    assert y.isfinite().all()
    check(x, codes, scales, None, y)


@pytest.mark.parametrize("M", TOKENS)
def test_one_largest_input(M):
    """The largest finite input, alone in its token, reads one weight each."""
    say(f"w4 largest input M={M}")
    N, K, G = 64, 256, 64
    codes, scales = codes_scales(N, K, G, M + 2)
    scales = torch.full_like(scales, 2.0 ** -9)
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    at = torch.arange(M, device="cuda") * 37 % K
    big = torch.finfo(BF).max
    x[torch.arange(M, device="cuda"), at] = big
    w4, s = B.w4_pack_weight(codes, scales)
    want = (codes.t()[at].double() * 2.0 ** -9 * big).float().to(BF)
    assert torch.equal(B.w4_linear(x, w4, s), want)

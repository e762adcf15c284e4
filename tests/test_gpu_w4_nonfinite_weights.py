"""Weights that are not finite, through the 4-bit converter and the linear."""
from __future__ import annotations

import pytest

from tests.test_gpu_w4 import gen, say, unpacked
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


@pytest.mark.parametrize("G", [32, 64, 128])
def test_weights_that_are_not_finite(G):
    """A group that holds a NaN has a NaN scale, one that holds an Inf an
    infinite one, other groups are as before, and the channel's outputs are
    not finite."""
    say(f"w4 not finite G={G}")
    N, K = 48, 384
    w = torch.randn(N, K, generator=gen(G), device="cuda").to(BF)
    c0, s0 = unpacked(*B.w4_quantize_weight(w, group=G))
    # a NaN at each place of a lane's eight inputs, of its four chunks and of
    # the four lanes of a channel, one to a channel; then Infs, then both
    bad = [(i, 37 * i % K, float("nan")) for i in range(32)]
    bad += [(33, 200, float("inf")), (34, 37, -float("inf"))]
    for n, k, v in bad:
        w[n, k] = v
    w[47, 300:302] = torch.tensor([float("inf"), float("nan")])
    w4, s4 = B.w4_quantize_weight(w, group=G)
    c, s = unpacked(w4, s4)
    rest = torch.ones(N, K // G, dtype=torch.bool)
    for n, k, v in bad:
        got = s[n, k // G]
        assert got.isnan() if v != v else got == float("inf"), (n, k)
        rest[n, k // G] = False
    assert s[47, 300 // G].isnan()
    rest[47, 300 // G] = False
    assert torch.equal(s[rest].view(torch.int16), s0[rest].view(torch.int16))
    kept = rest.repeat_interleave(G, 1)
    assert torch.equal(c[kept], c0[kept])
    rows = sorted({n for n, _, _ in bad} | {47})
    fine = [n for n in range(N) if n not in rows]
    for M in (3, 20):
        y = B.w4_linear(torch.ones(M, K, dtype=BF, device="cuda"), w4, s4)
        assert not y[:, rows].isfinite().any()
        assert y[:, fine].isfinite().all()

"""Batches of sequences without keys."""
from __future__ import annotations

import pytest

from tests.test_gpu_attention import rand, gen
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


@pytest.mark.parametrize("Bn,Lq", [(1, 5), (3, 1), (3, 5), (2, 300)])
def test_a_batch_without_keys_gives_zeros(Bn, Lq):
    q = rand(gen(1), Bn, Lq, 4, 64)
    cache = rand(gen(2), Bn, 40, 2, 64)
    lens = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    none = torch.empty(Bn, 0, 2, 64, dtype=BF, device="cuda")
    for k, kw in ((none, {}), (cache[:, :0], {}), (cache[:, 7:7], {}),
                  (none, dict(k_lens=lens))):
        out = torch.full_like(q, 7.0)
        assert B.attention(q, k, k, out=out, **kw) is out
        assert (out == 0).all()

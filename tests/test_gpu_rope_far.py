"""Rotary tables at positions up to the ends of INT32 against 60 digits: the
angle's error is within what the header states."""
from __future__ import annotations

import pytest

from tests import headref as R
from tests import ropeexact as X
from w8a8_int8_gemm_amd import binding as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("kw", [
    dict(), dict(theta=5e5), dict(theta=1e12), dict(theta=1e100),
    dict(scaling="linear", factor=3.7), dict(scaling="ntk", factor=1e5),
    dict(scaling="yarn", factor=40.0, original=4096.0, amplitude=1.25)])
@pytest.mark.parametrize("kind", ["int32", "float32"])
@pytest.mark.parametrize("P", [60, 64, 127])
def test_far_positions(P, kind, kw):
    at = [2**31 - 1, -2**31, 1234567891, -987654321, 2**24 + 1, 1000003, 77]
    if kind == "float32":
        at = [float(torch.tensor(float(a)).float()) for a in at] + [2.0**40 + 2**18]
    pos = torch.tensor(at, dtype=getattr(torch, kind), device="cuda")
    got = B.rope_table(pos, P, **kw).double().cpu()
    kw = dict(kw)
    amplitude = kw.pop("amplitude", 1.0)
    f = X.frequencies(P, **kw)
    want = [[X.turned(a, v) for v in f] for a in at]
    cos, sin, size = (torch.tensor([[w[i] for w in row] for row in want],
                                   dtype=torch.float64) for i in range(3))
    # the reference's own 2^-51 and what the header allows
    bound = amplitude * (1.75 * 2.0 ** -52 * size + 6 * R.U + 2.0 ** -51)
    for i, w in enumerate((cos, sin)):
        off = (got[:, i] - amplitude * w).abs() / bound
        assert off.max() <= 1, (i, off.max().item(), off.argmax().item())

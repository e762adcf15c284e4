"""The stages of a NormedBlock between its projections, against the oracle on
the buffers that the stage before left: the quantization of V's output, SiLU
and SwiGLU, and post-norms with weights and biases."""
from __future__ import annotations

import pytest

import oracle
from tests import normref as R
from tests.test_gpu_normed_block import make, ref_kw, shapes
from w8a8_int8_gemm_amd import block as BL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


def activated(t, mlp):
    orc = oracle.default()
    bits = BL.from_device_bf16(t)
    return orc.swiglu_bf16(bits) if mlp == "swiglu" else orc.silu_bf16(bits)


def same_codes(bits, q, s):
    want_q, want_s = oracle.default().quantize_act(bits)
    assert (q.cpu().numpy() == want_q).all()
    assert (s.cpu().numpy() == want_s).all()


@pytest.mark.parametrize("mlp", ["silu", "swiglu"])
@pytest.mark.parametrize("M", [5, 300])
def test_int8_stages(M, mlp):
    projs = shapes(256, 384, 512, mlp)
    x, n, dev = make(M, projs, "rms", "rms", 3)
    blk = BL.NormedBlock(M, projs, mlp)
    blk.run(x, dev, n)
    same_codes(BL.from_device_bf16(blk.out["v"]), blk.oq, blk.os)
    same_codes(activated(blk.out["fc1"], mlp), blk.hq, blk.hs)


@pytest.mark.parametrize("mlp", ["silu", "swiglu"])
@pytest.mark.parametrize("M", [1, 13])
def test_four_bit_stages(M, mlp):
    projs = shapes(256, 384, 512, mlp)
    x, n, dev = make(M, projs, "rms", "rms", 4, padded=False)
    four = {k: BL.to_four_bit(p, 128) for k, p in dev.items()}
    blk = BL.NormedBlock(M, projs, mlp, four_bit=True)
    blk.run(x, four, n)
    assert (BL.from_device_bf16(blk.h) == activated(blk.out["fc1"], mlp)).all()


@pytest.mark.parametrize("four_bit", [False, True])
def test_post_layer_norm_with_biases(four_bit):
    M, projs = 37, shapes(256, 384, 512, "silu")
    x, n, dev = make(M, projs, "layer", "layer", 5)
    g = torch.Generator("cuda").manual_seed(6)
    n.post_bias = tuple(torch.randn(256, generator=g, device="cuda").to(
        torch.bfloat16) for _ in "am")
    if four_bit:
        dev = {k: BL.to_four_bit(p, 32) for k, p in dev.items()}
    blk = BL.NormedBlock(M, projs, four_bit=four_bit)
    out = blk.run(x, dev, n)
    r, y = R.block(x, **ref_kw(n, 0, blk.out["o"], 1))
    R.check_bf16(blk.r, *r)
    if four_bit:
        R.check_bf16(blk.y, *y)
    else:
        R.check_codes(blk.yq, blk.ys, *y)
    R.check_bf16(out, *R.block(blk.r, **ref_kw(n, 1, blk.out["fc2"]))[0])
    dead = n.mod_row < 0
    assert torch.equal(out[dead], x[dead])

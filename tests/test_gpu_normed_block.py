"""A block's norms, projections, gates and residuals run together, as INT8 and
as 4-bit projections: every stage against its definition on the buffers that
the stage before it left."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from tests import normref as R
from tests.test_gpu_w4 import check as check_w4
from tests.test_gpu_w4 import unpacked
from w8a8_int8_gemm_amd import block as BL
from w8a8_int8_gemm_amd import datagen as D

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16


def shapes(H, A, F, mlp):
    fc1 = 2 * F if mlp == "swiglu" else F
    return (D.Proj("q", 0, A, H), D.Proj("k", 1, A, H), D.Proj("v", 2, A, H),
            D.Proj("o", 3, H, A), D.Proj("fc1", 4, fc1, H),
            D.Proj("fc2", 5, H, F))


def make(M, projs, norm, post, seed, padded=True):
    g = torch.Generator("cuda").manual_seed(seed)
    H = projs[0].K
    rand = lambda *s, std=1.0, mean=0.0: (
        mean + std * torch.randn(*s, generator=g, device="cuda")).to(BF)
    x = rand(M, H)
    pair = lambda mean: (rand(H, mean=mean, std=0.1), rand(H, mean=mean, std=0.1))
    row = torch.arange(M, device="cuda", dtype=torch.int32) * 3 // M
    if padded:
        row[M - M // 4:] = -1
    n = BL.BlockNorms(rand(3, 6 * H, std=0.3), row, norm=norm,
                      weight=pair(1.0),
                      bias=pair(0.0) if norm == "layer" else (None, None),
                      post_norm=post,
                      post_weight=pair(1.0) if post != "none" else (None, None),
                      residual_scale=0.75)
    dev = {p.name: BL.upload_proj(p, D.proj_params(p, seed)) for p in projs}
    return x, n, dev


def ref_kw(n, side, branch=None, nxt=None):
    kw = dict(mod_row=n.mod_row)
    if branch is not None:
        b = n.behind(side)
        b["post_norm"] = b.pop("post_norm")
        kw.update(branch=branch, **b)
    if nxt is not None:
        p = n.before(nxt)
        kw.update(norm_kind=p.pop("norm"), **p)
    return kw


def gemm_ref(q, s, p):
    orc = oracle.default()
    acc = orc.gemm_i32(q.cpu().numpy(), p.w.cpu().numpy())
    _, y = orc.epilogue(acc, s.cpu().numpy(), p.sw.cpu().numpy(),
                     BL.from_device_bf16(p.bias))
    return BL.to_device_bf16(y)


@pytest.mark.parametrize("M,norm,post,mlp", [
    (300, "rms", "none", "silu"), (37, "layer", "rms", "swiglu")])
def test_int8_block(M, norm, post, mlp):
    projs = shapes(256, 384, 512, mlp)
    x, n, dev = make(M, projs, norm, post, 5)
    blk = BL.NormedBlock(M, projs, mlp)
    # the codes of the first norm are overwritten by the second: keep them
    first = BL.B.norm_modulate_quantize(x, **n.before(0), mod_row=n.mod_row)
    out = blk.run(x, dev, n)
    R.check_codes(*first, *R.block(x, **ref_kw(n, 0, nxt=0))[1])
    for name in ("q", "k", "v"):
        assert torch.equal(blk.out[name], gemm_ref(*first, dev[name])), name
    assert torch.equal(blk.out["o"], gemm_ref(blk.oq, blk.os, dev["o"]))
    r, y = R.block(x, **ref_kw(n, 0, blk.out["o"], 1))
    R.check_bf16(blk.r, *r)
    R.check_codes(blk.yq, blk.ys, *y)
    assert torch.equal(blk.out["fc1"], gemm_ref(blk.yq, blk.ys, dev["fc1"]))
    assert torch.equal(blk.out["fc2"], gemm_ref(blk.hq, blk.hs, dev["fc2"]))
    R.check_bf16(out, *R.block(blk.r, **ref_kw(n, 1, blk.out["fc2"]))[0])
    dead = n.mod_row < 0
    assert torch.equal(out[dead], x[dead])


@pytest.mark.parametrize("M,norm,post,mlp", [
    (1, "rms", "none", "silu"), (13, "layer", "rms", "swiglu"),
    (50, "rms", "rms", "silu")])
def test_four_bit_block(M, norm, post, mlp):
    projs = shapes(256, 384, 512, mlp)
    x, n, dev = make(M, projs, norm, post, 6, padded=M > 4)
    four = {k: BL.to_four_bit(p, 64) for k, p in dev.items()}
    blk = BL.NormedBlock(M, projs, mlp, four_bit=True)
    first = BL.B.norm_modulate(x, **n.before(0), mod_row=n.mod_row)
    out = blk.run(x, four, n)
    R.check_bf16(first, *R.block(x, **ref_kw(n, 0, nxt=0))[1])

    def linear(a, name):
        p = four[name]
        codes, scales = unpacked(p.w4, p.w4_scale)
        check_w4(a, codes.cuda(), scales.cuda(), p.bias, blk.out[name])
    for name in ("q", "k", "v"):
        linear(first, name)
    linear(blk.out["v"], "o")
    r, y = R.block(x, **ref_kw(n, 0, blk.out["o"], 1))
    R.check_bf16(blk.r, *r)
    R.check_bf16(blk.y, *y)
    linear(blk.y, "fc1")
    linear(blk.h, "fc2")
    R.check_bf16(out, *R.block(blk.r, **ref_kw(n, 1, blk.out["fc2"]))[0])


@pytest.mark.parametrize("four_bit", [False, True])
def test_block_in_a_graph(four_bit):
    """Captured once; replays with new inputs equal the eager run, with eager
    runs of another block in between."""
    M, projs = 21, shapes(256, 256, 512, "silu")
    x, n, dev = make(M, projs, "rms", "rms", 7)
    if four_bit:
        dev = {k: BL.to_four_bit(p, 32) for k, p in dev.items()}
    blk, other = (BL.NormedBlock(M, projs, four_bit=four_bit) for _ in "ab")
    y = torch.empty_like(x)
    blk.run(x, dev, n, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.run(x, dev, n, out=y)
    for i in range(3):
        x.copy_(torch.randn(x.shape, device="cuda", generator=torch.Generator(
            "cuda").manual_seed(i)))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, other.run(x, dev, n))


def test_int8_block_at_model_width():
    """One block at width 5376 and 4096 tokens: its norms against 64 bits."""
    M = 4096
    projs = D.BLOCK_PROJS
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(M, 5376, device="cuda", generator=g).to(BF)
    n = BL.BlockNorms((0.3 * torch.randn(4, 6 * 5376, device="cuda",
                                         generator=g)).to(BF),
                      torch.arange(M, device="cuda", dtype=torch.int32) // 1024,
                      post_norm="rms")
    dev = {}
    for p in projs:
        w = torch.randint(-127, 128, (p.N, p.K), device="cuda", generator=g,
                          dtype=torch.int8)
        sw = torch.exp(torch.randn(p.N, device="cuda", generator=g) * 0.3 - 6)
        dev[p.name] = BL.DeviceProj(p.name, p.N, p.K, w, sw, torch.zeros(
            p.N, dtype=BF, device="cuda"))
    blk = BL.NormedBlock(M, projs)
    out = blk.run(x, dev, n)
    r, y = R.block(x, **ref_kw(n, 0, blk.out["o"], 1))
    R.check_bf16(blk.r, *r)
    R.check_codes(blk.yq, blk.ys, *y)
    R.check_bf16(out, *R.block(blk.r, **ref_kw(n, 1, blk.out["fc2"]))[0])
    rows = np.array([0, 1, 255, 256, 4095])
    at = torch.from_numpy(rows).cuda()
    assert torch.equal(blk.out["fc2"][at], gemm_ref(
        blk.hq[at], blk.hs[at], dev["fc2"]))

"""The rotary table, the head norms with rotation and the attention run together
in a block, as INT8 and as 4-bit projections, to the block's own tokens and to
other states: every stage against its definition on the buffers that the stage
before it left."""
from __future__ import annotations

import pytest

from tests import headref as HR
from tests import normref as R
from tests.test_gpu_normed_block import gemm_ref, make, ref_kw
from tests.test_gpu_w4 import check as check_w4
from tests.test_gpu_w4 import unpacked
from w8a8_int8_gemm_amd import block as BL
from w8a8_int8_gemm_amd import datagen as D

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

BF = torch.bfloat16
B = BL.B
W = 64  # a head's width


def shapes(H, heads, k_heads, F, C=None):
    C = H if C is None else C
    return (D.Proj("q", 0, heads * W, H), D.Proj("k", 1, k_heads * W, C),
            D.Proj("v", 2, k_heads * W, C), D.Proj("o", 3, H, heads * W),
            D.Proj("fc1", 4, F, H), D.Proj("fc2", 5, H, F))


def vec(seed, *s):
    g = torch.Generator("cuda").manual_seed(seed)
    return (1 + 0.2 * torch.randn(*s, generator=g, device="cuda")).to(BF)


def heads_of(M, positions=None, **kw):
    h = BL.BlockHeads(W, q_weight=vec(1, W), k_weight=vec(2, W), **kw)
    if positions is not None:
        h.table = B.rope_table(positions, (16, 8, 8))
    return h


def positions(M):
    """Frame, row and column of every token."""
    m = torch.arange(M, device="cuda", dtype=torch.int32)
    return torch.stack([m // 30, m // 6 % 5, m % 6], 1).contiguous()


def check_attention(blk, h, q, k, v, spans):
    """From the projections' outputs q, k, v to what the block left."""
    cut = lambda t: t.unflatten(1, (-1, W))
    table = None if blk.context_tokens is not None else h.table
    R.check_bf16(cut(blk.out["q"]), *HR.heads(
        cut(q), h.norm, h.q_weight, table=table, row=h.row))
    R.check_bf16(cut(blk.out["k"]), *HR.heads(
        cut(k), h.norm, h.k_weight, table=table, row=h.row))
    assert torch.equal(blk.out["v"], v)
    want, bound, covered = HR.attention(
        cut(blk.out["q"]), cut(blk.out["k"]), cut(v), spans, h.scale)
    R.check_bf16(cut(blk.a)[covered], want[covered], bound[covered])


@pytest.mark.parametrize("M,kv,seqs", [(300, 6, 1), (300, 2, 3), (37, 2, 1)])
def test_int8_block_to_its_own_tokens(M, kv, seqs):
    projs = shapes(256, 6, kv, 512)
    x, n, dev = make(M, projs, "rms", "none", 5, padded=False)
    h = heads_of(M, positions(M), batch=seqs)
    blk = BL.NormedBlock(M, projs, heads=h)
    first = B.norm_modulate_quantize(x, **n.before(0), mod_row=n.mod_row)
    out = blk.run(x, dev, n)
    q, k, v = (gemm_ref(*first, dev[name]) for name in "qkv")
    check_attention(blk, h, q, k, v, HR.sequences(M, M, seqs))
    codes = B.quantize_act(blk.a)
    assert torch.equal(codes[0], blk.oq) and torch.equal(codes[1], blk.os)
    assert torch.equal(blk.out["o"], gemm_ref(blk.oq, blk.os, dev["o"]))
    r, y = R.block(x, **ref_kw(n, 0, blk.out["o"], 1))
    R.check_bf16(blk.r, *r)
    R.check_codes(blk.yq, blk.ys, *y)
    R.check_bf16(out, *R.block(blk.r, **ref_kw(n, 1, blk.out["fc2"]))[0])


def test_int8_block_with_padding_tokens():
    """The norms' padding tokens at the end are left out of the keys."""
    M = 200
    projs = shapes(256, 4, 4, 512)
    x, n, dev = make(M, projs, "layer", "rms", 6)
    live = int((n.mod_row >= 0).sum())
    assert live < M
    h = heads_of(M, positions(M), k_lens=torch.tensor(
        [live], dtype=torch.int32, device="cuda"))
    blk = BL.NormedBlock(M, projs, heads=h)
    out = blk.run(x, dev, n)
    first = B.norm_modulate_quantize(x, **n.before(0), mod_row=n.mod_row)
    q, k, v = (gemm_ref(*first, dev[name]) for name in "qkv")
    check_attention(blk, h, q, k, v, HR.sequences(M, M, 1, k_lens=h.k_lens))
    assert torch.equal(out[live:], x[live:])


@pytest.mark.parametrize("M,Mk", [(300, 77), (5, 200)])
@pytest.mark.parametrize("four_bit", [False, True])
def test_block_to_other_states(M, Mk, four_bit):
    projs = shapes(256, 4, 2, 512, C=384)
    x, n, dev = make(M, projs, "rms", "none", 7, padded=False)
    g = torch.Generator("cuda").manual_seed(8)
    ctx = torch.randn(Mk, 384, generator=g, device="cuda").to(BF)
    lens = torch.tensor([Mk - 20], dtype=torch.int32, device="cuda")
    h = heads_of(M, k_lens=lens)
    blk = BL.NormedBlock(M, projs, heads=h, context_tokens=Mk,
                         four_bit=four_bit)
    if four_bit:
        four = {name: BL.to_four_bit(p) for name, p in dev.items()}
        first = B.norm_modulate(x, **n.before(0), mod_row=n.mod_row)
        q, k, v = (B.w4_linear(a, four[name].w4, four[name].w4_scale,
                               four[name].bias)
                   for a, name in ((first, "q"), (ctx, "k"), (ctx, "v")))
        blk.run(x, four, n, context=ctx)
        p = four["o"]
        codes, scales = unpacked(p.w4, p.w4_scale)
        check_w4(blk.a, codes.cuda(), scales.cuda(), p.bias, blk.out["o"])
    else:
        first = B.norm_modulate_quantize(x, **n.before(0), mod_row=n.mod_row)
        codes = B.quantize_act(ctx)
        q, k, v = (gemm_ref(*a, dev[name]) for a, name in (
            (first, "q"), (codes, "k"), (codes, "v")))
        blk.run(x, dev, n, context=ctx)
        assert torch.equal(blk.out["o"], gemm_ref(blk.oq, blk.os, dev["o"]))
    check_attention(blk, h, q, k, v, HR.sequences(M, Mk, 1, k_lens=lens))


def test_block_in_a_graph():
    """Captured once with the table of its positions; replays with new inputs
    and positions equal the eager run."""
    M = 90
    projs = shapes(256, 4, 2, 256)
    x, n, dev = make(M, projs, "rms", "rms", 9, padded=False)
    pos = positions(M)
    h = heads_of(M, pos)
    blk, other = (BL.NormedBlock(M, projs, heads=h) for _ in "ab")
    y = torch.empty_like(x)

    def step(b, out=None):
        B.rope_table(pos, (16, 8, 8), out=h.table)
        return b.run(x, dev, n, out=out)
    step(blk, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(blk, y)
    for i in range(3):
        x.copy_(torch.randn(x.shape, device="cuda", generator=torch.Generator(
            "cuda").manual_seed(i)))
        pos.add_(7)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, step(other))


def test_block_refuses():
    projs = shapes(256, 4, 2, 256)
    with pytest.raises(ValueError):
        BL.NormedBlock(8, projs, context_tokens=9)
    with pytest.raises(ValueError):
        BL.NormedBlock(8, projs, heads=heads_of(8, positions(8)),
                       context_tokens=9)
    x, n, dev = make(8, projs, "rms", "none", 1, padded=False)
    ctx = torch.zeros(9, 256, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        BL.NormedBlock(8, projs).run(x, dev, n, context=ctx)
    with pytest.raises(ValueError):
        BL.NormedBlock(8, projs, heads=heads_of(8), context_tokens=9).run(
            x, dev, n)

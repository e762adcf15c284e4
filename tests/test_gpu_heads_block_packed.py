"""Blocks whose sequences lie packed and leave some tokens out: every run gives
those tokens the same, whatever the buffers held before."""
from __future__ import annotations

import pytest

from tests import headref as HR
from tests.test_gpu_heads_block import (check_attention, heads_of, positions,
                                        shapes)
from tests.test_gpu_normed_block import gemm_ref, make
from w8a8_int8_gemm_amd import block as BL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

B = BL.B
BF = torch.bfloat16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# First and last tokens outside, an empty sequence, tokens behind the last one.
SPANS = [([0, 90, 250], None), ([0, 90, 90, 300], None),
         ([3, 40, 40, 211], [0, 100, 110, 280]), ([0, 0, 0], [0, 150, 300]),
         ([0, 33], None)]


def uncovered(M, offsets):
    out = torch.ones(M, dtype=torch.bool, device="cuda")
    out[offsets[0]:offsets[-1]] = False
    return out


@pytest.mark.parametrize("qo,ko", SPANS)
@pytest.mark.parametrize("four_bit", [False, True])
def test_tokens_of_no_sequence(qo, ko, four_bit):
    M = 300
    projs = shapes(256, 6, 2, 512)
    x, n, dev = make(M, projs, "rms", "none", 21, padded=False)
    if four_bit:
        dev = {name: BL.to_four_bit(p) for name, p in dev.items()}
    h = heads_of(M, positions(M), q_offsets=ints(qo),
                 k_offsets=ints(qo if ko is None else ko))
    blk, other = (BL.NormedBlock(M, projs, heads=h, four_bit=four_bit)
                  for _ in "ab")
    # what memory may hold before a block's first run
    blk.a.fill_(float("nan"))
    other.a.fill_(31.0)
    got = blk.run(x, dev, n).clone()
    a = blk.a.clone()
    outside = uncovered(M, qo)
    assert (a[outside] == 0).all() and got.isfinite().all()
    assert torch.equal(other.run(x, dev, n), got)
    # a run on other tokens in between leaves nothing behind
    blk.run(torch.randn_like(x.float()).to(BF), dev, n)
    h.q_offsets = ints([0] + [M] * (len(qo) - 1))
    blk.run(x, dev, n)
    h.q_offsets = ints(qo)
    assert torch.equal(blk.run(x, dev, n), got)
    assert torch.equal(blk.a, a)


@pytest.mark.parametrize("qo,ko", SPANS)
def test_packed_block_against_its_definition(qo, ko):
    M = 300
    projs = shapes(256, 4, 4, 512)
    x, n, dev = make(M, projs, "layer", "rms", 22, padded=False)
    h = heads_of(M, positions(M), q_offsets=ints(qo),
                 k_offsets=ints(qo if ko is None else ko))
    blk = BL.NormedBlock(M, projs, heads=h)
    first = B.norm_modulate_quantize(x, **n.before(0), mod_row=n.mod_row)
    blk.run(x, dev, n)
    q, k, v = (gemm_ref(*first, dev[name]) for name in "qkv")
    check_attention(blk, h, q, k, v, HR.sequences(
        M, M, len(qo) - 1, h.q_offsets, h.k_offsets))


def test_on_another_stream_and_in_a_graph():
    M, qo = 200, [5, 60, 171]
    projs = shapes(256, 4, 2, 256)
    x, n, dev = make(M, projs, "rms", "none", 23, padded=False)
    h = heads_of(M, positions(M), q_offsets=ints(qo), k_offsets=ints(qo))
    want = BL.NormedBlock(M, projs, heads=h).run(x, dev, n)
    blk = BL.NormedBlock(M, projs, heads=h)
    blk.a.fill_(float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = blk.run(x, dev, n, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    y = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.run(x, dev, n, out=y)
    for i in range(3):
        x.copy_(torch.randn_like(x.float()).to(BF))
        blk.a.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, BL.NormedBlock(M, projs, heads=h).run(x, dev, n))

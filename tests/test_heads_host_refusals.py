"""What the binding and the block make of their arguments before the library is
called, on the host (the check that a tensor lies on the GPU is left out)."""
from __future__ import annotations

import pytest
import torch

from tests.test_heads_host import ARG, DEVICE, attend, no_gpu
from w8a8_int8_gemm_amd import binding as B
from w8a8_int8_gemm_amd import block as BL
from w8a8_int8_gemm_amd import datagen as D

BF = torch.bfloat16


@pytest.fixture
def anywhere(monkeypatch):
    monkeypatch.setattr(B, "_on_current_gpu", lambda t, name: None)


def test_a_batch_without_rows(anywhere):
    """Sequences of no rows follow each other at any stride."""
    for t in (torch.zeros(3, 0, 2, 64, dtype=BF),
              torch.zeros(3, 7, 2, 64, dtype=BF)[:, :0],
              torch.zeros(3, 7, 4, 64, dtype=BF)[:, 4:4, :2]):
        assert B._head_rows(t, "k", True) == (0, 128)
    assert B._head_rows(torch.zeros(0, 2, 64, dtype=BF), "k", True) == (0, 128)
    # rows that do not follow each other are refused as before
    with pytest.raises(ValueError, match="follow each other"):
        B._head_rows(torch.zeros(3, 7, 2, 64, dtype=BF)[:, :5], "k", True)


@pytest.mark.parametrize("weight", [
    torch.ones(5, 64, dtype=BF), torch.ones(2, 64, dtype=BF),
    torch.ones(0, 64, dtype=BF), torch.ones(1, 64),
    torch.ones(1, 128, dtype=BF)[:, ::2], torch.ones(1, 1, 64, dtype=BF)])
@pytest.mark.parametrize("name", ["q_weight", "q_bias", "k_weight", "k_bias"])
def test_vectors_of_one_head(anywhere, monkeypatch, name, weight):
    """One head takes [1, width] or [width], and no vectors of other heads."""
    x = torch.zeros(3, 1, 64, dtype=BF)
    kw = dict(norm="layer", out=(x.clone(), x.clone()))
    with pytest.raises(ValueError, match=name.replace("_", " ")):
        B.head_norm_rope(x, x, **{name: weight}, **kw)
    with pytest.raises(TypeError, match=name.replace("_", " ")):
        B.head_norm_rope(x, x, **{name: [1.0] * 64}, **kw)
    one = torch.ones(1, 64, dtype=BF)
    for t in (one, one[0]):
        arg, _ = B._heads_arg(x, None, 2, t, t, 1e-6, "q")
        assert (arg.norm.weight, arg.per_head) == (t.data_ptr(), 0)
    # [1, width] beside [width] stays allowed where they mean the same
    arg, _ = B._heads_arg(x, None, 2, one, one[0], 1e-6, "q")
    assert (arg.norm.weight, arg.norm.bias) == (one.data_ptr(),) * 2


MOST = (2.0 - 2.0 ** -23) * 2.0 ** 127  # binary32's largest


def test_scales_past_the_range_are_refused():
    """The kernel multiplies scores by scale * log2(e)."""
    for scale in (MOST, 2.0 ** 127.5, MOST / 1.4426):
        assert attend(scale=scale) == ARG


@no_gpu
def test_scales_of_the_range_are_taken():
    for scale in (MOST / 1.4428, 1.0, 2.0 ** -126, 2.0 ** -149):
        assert attend(scale=scale) == DEVICE


PROJS = (D.Proj("q", 0, 256, 128), D.Proj("k", 1, 128, 128),
         D.Proj("v", 2, 128, 128), D.Proj("o", 3, 128, 256),
         D.Proj("fc1", 4, 256, 128), D.Proj("fc2", 5, 128, 256))


@pytest.mark.parametrize("kw,context,message", [
    (dict(row=1), 9, "not turned"), (dict(row=1, table=1), 9, "not turned"),
    (dict(table=1), 9, "not turned"), (dict(row=1), None, "needs a table"),
    (dict(norm="none", q_weight=1), None, "need a norm"),
    (dict(norm="none", k_weight=1, table=1), None, "need a norm"),
    (dict(norm="none", k_bias=1), 9, "need a norm"),
    (dict(norm="none", q_bias=1), 9, "need a norm")])
def test_block_refuses_what_it_would_not_use(kw, context, message):
    make = lambda heads: BL.NormedBlock(8, PROJS, device="cpu", heads=heads,
                                        context_tokens=context)
    with pytest.raises(ValueError, match=message):
        make(BL.BlockHeads(64, **kw))
    # also where they are set behind the block's construction
    heads = BL.BlockHeads(64)
    block = make(heads)
    for name, value in kw.items():
        setattr(heads, name, value)
    with pytest.raises(ValueError, match=message):
        block._attend(None)

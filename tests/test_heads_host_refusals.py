"""What the binding and the block make of their arguments before the library is
called, on the host (the check that a tensor lies on the GPU is left out)."""
from __future__ import annotations

import pytest
import torch

from w8a8_int8_gemm_amd import binding as B

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

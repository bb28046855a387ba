"""Blocks of feedforward that cannot be trained say so.  No kernel runs here."""
from __future__ import annotations

import pytest
import torch

from warp_specialized_tma_gb300 import feedforward, ffn

bf = torch.bfloat16


def cpu(*shape):
    return torch.zeros(*shape, dtype=bf)


def test_a_block_that_keeps_nothing_is_not_trained(monkeypatch):
    block = feedforward.GatedFeedForward(cpu(16, 8), cpu(16, 8), cpu(8, 16), save=None)
    # gated() then returns h alone, whose two rows must not be taken for h and what was kept
    monkeypatch.setattr(ffn, "gated", lambda x, *rest, save=None: cpu(x.shape[0], 16))
    monkeypatch.setattr(ffn, "linear", lambda h, w, residual=None: cpu(len(h), 8))
    with pytest.raises(ValueError, match="keeps nothing"):
        block.forward_train(cpu(2, 8))
    assert block.forward(cpu(2, 8)).shape == (2, 8)


def test_what_a_block_keeps_is_checked():
    with pytest.raises(ValueError, match="save must be one of"):
        feedforward.GatedFeedForward(cpu(16, 8), cpu(16, 8), cpu(8, 16), save="fp8")

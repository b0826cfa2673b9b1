"""examples/hybrid_model.py with attention: what its caches cannot hold is refused, not left out."""
from __future__ import annotations

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
from hybrid_model import HybridModel, documents  # noqa: E402


def test_prompts_longer_than_the_caches():
    model = HybridModel(vocab=16, d=32, d_ff=32, blocks=1, fast=(), attend=(0,), max_seq_len=100, device="cpu")
    with pytest.raises(ValueError, match="max_seq_len=100"):
        model.prefill(torch.zeros(1, 128, dtype=torch.long))


@pytest.mark.gpu
def test_decoding_to_the_caches_end_and_no_further():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    model = HybridModel(vocab=64, blocks=2, fast=(), attend=(0,), max_seq_len=66)
    tokens, _, _ = documents(2, 128, 64, seed=5)
    model.prefill(tokens[:, :64])
    for t in (64, 65):
        assert torch.isfinite(model.decode(tokens[:, t])).all()
    with pytest.raises(ValueError, match="max_seq_len=66"):
        model.decode(tokens[:, 66])
    # a new prefill begins anew
    model.prefill(tokens[:, :64])
    assert torch.isfinite(model.decode(tokens[:, 64])).all()

"""Attention over prompts where something that is not finite is seen."""
from __future__ import annotations

import math

import pytest
import torch

from chunked_weight_mlp_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.load()


def rand(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [64, 128])
def test_a_value_far_below_the_maximum(dh, dtype, value):
    """Scores rise along the keys by half a unit each, so that the weight of an early key is less
    than any fp32 number for late queries: its value makes them NaN (infinite) all the same."""
    n, at = 700, 3
    q = torch.ones((n, 1, dh), dtype=dtype, device=DEV)
    k = (torch.arange(n, device=DEV, dtype=F32)[:, None, None] / 16 - 20).expand(n, 1, dh).to(dtype).contiguous()
    v = rand((n, 1, dh), 1, dtype)
    o, lse = A.attention_forward(q, k, v, scale=0.125)
    bad = v.clone()
    bad[at, 0, 5] = value
    oo, ll = A.attention_forward(q, k, bad, scale=0.125)
    assert not torch.isfinite(oo[at:, 0, 5]).any()
    keep = torch.arange(dh, device=DEV) != 5
    assert torch.equal(oo[..., keep], o[..., keep]) and torch.equal(oo[:at], o[:at]) and torch.equal(ll, lse)

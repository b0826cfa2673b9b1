"""Sizes that do not fit the C structures' 32 bits are refused by the Python operators, before
anything is computed (tensors of no memory)."""
from __future__ import annotations

import pytest
import torch

from chunked_weight_mlp_amd import attention as A
from chunked_weight_mlp_amd import ipttt as B

FAR = (2 ** 31, 2 ** 32 + 2)


def refused(call, *args, **kw):
    with pytest.raises(B.IptttError) as ei:
        call(*args, **kw)
    assert ei.value.status == B.IPTTT_E_INVALID and "32 bits" in str(ei.value), str(ei.value)


def wide(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("far", FAR)
def test_heads(far):
    q, k = torch.zeros(3, 2, 16), torch.zeros(3, 1, 16)
    refused(A.attention_forward, wide(3, far, 16), k, k)
    refused(A.attention_forward, wide(3, far, 16), wide(3, far, 16), wide(3, far, 16))
    refused(A.attention_forward, wide(1, 1, far), wide(1, 1, far), wide(1, 1, far))
    refused(A.attention_backward, q, wide(3, far, 16), wide(3, far, 16), q, torch.zeros(2, 3), q)
    op = A.HeadNorm(None, None, torch.zeros(4, dtype=torch.float64), head_dim=16, dtype=torch.float32)
    pos = torch.zeros(3, dtype=torch.int32)
    refused(op.forward, wide(3, far, 16), k, pos)
    refused(op.forward, q, wide(3, far, 16), pos)


@pytest.mark.parametrize("far", FAR)
def test_head_norm(far):
    f = torch.zeros(4, dtype=torch.float64)
    refused(A.HeadNorm, None, None, f, head_dim=far, dtype=torch.float32)
    refused(A.HeadNorm, None, None, wide(far // 2, dtype=torch.float64), head_dim=16, dtype=torch.float32)


@pytest.mark.parametrize("far", FAR)
def test_offsets(far):
    q, k = torch.zeros(3, 2, 16), torch.zeros(3, 1, 16)
    off = wide(far + 1, dtype=torch.int32)
    refused(A.attention_forward, q, k, k, off)


@pytest.mark.parametrize("far", FAR)
def test_cache_and_table(far):
    for shape in ((far, 1, 8, 16), (1, far, 8, 16), (1, 1, far, 16), (1, 1, 8, far)):
        refused(A.KVCache, wide(*shape), wide(*shape))
    pages = torch.zeros(4, 1, 8, 16)
    cache = A.KVCache(pages, pages.clone())
    q, lens = torch.zeros(3, 2, 16), torch.ones(3, dtype=torch.int32)
    refused(A.attention_step, q, cache, wide(3, far, dtype=torch.int32), lens)
    refused(A.attention_step, q, cache, wide(far, 2, dtype=torch.int32), lens)

"""Windows longer than any sequence, to the largest number of 32 bits, also where there are more
queries than keys: the results are those of no window."""
from __future__ import annotations

import pytest
import torch

import attention_reference as R
from chunked_weight_mlp_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.load()


def rand(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 30 + 1, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lq,lk", [([100], [40]), ([10, 300], [5, 200]), ([300], [1]), ([400, 7], [650, 7]), ([9], [0])])
def test_window_without_an_end(lq, lk, dtype, window):
    hq, hk, dh = 2, 1, 64
    q, dy = rand((sum(lq), hq, dh), 1, dtype, 2.0), rand((sum(lq), hq, dh), 4, dtype)
    k, v = rand((sum(lk), hk, dh), 2, dtype), rand((sum(lk), hk, dh), 3, dtype)
    at = dict(offsets=offsets(lq), k_offsets=offsets(lk))
    o, lse = A.attention_forward(q, k, v, window=window, **at)
    want, want_lse = A.attention_forward(q, k, v, **at)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    exact, _, bound, _ = R.attention(q, k, v, lq, lk, True, window)
    assert ((o.double() - exact).abs() <= bound).all()
    got = A.attention_backward(q, k, v, o, lse, dy, window=window, **at)
    want = A.attention_backward(q, k, v, o, lse, dy, **at)
    assert all(torch.equal(got[x], want[x]) for x in want)

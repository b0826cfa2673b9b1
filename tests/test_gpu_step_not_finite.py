"""The attention step where q, or keys and values that are seen, hold something that is not finite:
each result is of the formula's class (not_finite_reference.agree), whether one block has the
sequence or many share it."""
from __future__ import annotations

import math

import pytest
import torch

import not_finite_reference as N
from chunked_weight_mlp_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
PAGE = 32


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.load()


def rand(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def one(length, dtype, hq=4, hk=2, dh=64, std=2.0):
    """A cache with one sequence in pages of 32, its table, length and query. A length of 64 is
    one block's; the steps of longer ones are shared."""
    pages = -(-length // PAGE)
    cache = A.KVCache(rand((pages, hk, PAGE, dh), 1, dtype), rand((pages, hk, PAGE, dh), 2, dtype))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    return cache, table, torch.tensor([length], dtype=torch.int32, device=DEV), rand((1, hq, dh), 3, dtype, std)


def check(name, q, cache, length, dtype, o):
    hq, dh = q.shape[1:]
    for h in range(hq):
        g = h // (hq // cache.k_heads)
        k, v = (t[:, g].reshape(-1, dh)[:length] for t in (cache.k, cache.v))
        ok = torch.ones((1, length), dtype=torch.bool, device=DEV)
        want, _, bound, _ = N.forward(q[:, h], k, v, ok, dh ** -0.5, dtype)
        N.agree(f"{name}, head {h}", o[:, h], want, bound)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("what", ["k", "v", "q", "key", "keys"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("std", [2.0, 60.0])
@pytest.mark.parametrize("length", [64, 1500, 1501])
def test_class_of_results(length, std, dtype, what, value):
    """One channel of a key or a value, of the query; a whole key; the 64 keys of two pages. Of the
    channel's partners all are positive: a key of minus infinity has that score. At std 60 most
    weights are less than any fp32 number."""
    cache, table, lens, q = one(length, dtype, std=std)
    q[..., 7] = q[..., 7].abs() + 0.5
    cache.k[..., 7] = cache.k[..., 7].abs() + 0.5
    page = 0 if length == 64 else 20
    if what == "k":
        cache.k[page, 1, 9, 7] = value
    elif what == "v":
        cache.v[page, 1, 9, 7] = value
    elif what == "q":
        q[0, 2, 7] = value
    elif what == "key":
        cache.k[page, 1, 9] = value
    else:
        cache.k[page:page + 2, 1, :, 7] = value
    o = A.attention_step(q, cache, table, lens)
    check(f"{what} {value}", q, cache, length, dtype, o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("length", [64, 1500])
def test_keys_of_no_weight(length, dtype):
    """Keys whose score is minus infinity count as those that are not there do; if every key's is,
    the result is NaN; a value that is not finite makes NaN also where its weight is zero."""
    cache, table, lens, q = one(length, dtype)
    q[..., 7] = q[..., 7].abs() + 0.5
    page = 1 if length == 64 else 20
    without = table.clone()
    without[0, page] = -1
    want = A.attention_step(q, cache, without, lens)
    cache.k[page, :, :, 7] = -math.inf
    assert torch.equal(A.attention_step(q, cache, table, lens), want)
    cache.v[page, 0, 3, 11] = math.nan
    o = A.attention_step(q, cache, table, lens)
    assert torch.isnan(o[0, :2, 11]).all()
    o[0, :2, 11] = want[0, :2, 11]
    assert torch.equal(o, want)
    cache.k[:, 1, :, 7] = -math.inf
    o = A.attention_step(q, cache, table, lens)
    assert torch.isnan(o[0, 2:]).all() and torch.isfinite(o[0, :2, :11]).all()


def test_lse_of_keys_without_weight():
    """The C entry's log sum where no key has weight is minus infinity or NaN, in one block and
    shared."""
    for length in (64, 1500):
        cache, table, lens, q = one(length, F32)
        q[..., 7] = q[..., 7].abs() + 0.5
        cache.k[..., 7] = -math.inf
        o, lse = torch.empty_like(q), torch.zeros((1, 4), device=DEV)
        desc, tab = A.StepDesc(4, 0, 0.125), cache.table(table)
        need = A.ipttt_attention_step_workspace_bytes(desc, cache.desc, tab)
        ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
        A.ipttt_attention_step(desc, A._heads("q", q, q.shape, F32, q.device), cache.desc, tab, lens,
                               A._heads("o", o, q.shape, F32, q.device), lse, ws, need)
        assert torch.isnan(o).all() and (torch.isnan(lse) | (lse == -math.inf)).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("length", [64, 1500])
def test_a_scale_of_zero(length, dtype, value):
    """0 x infinity and 0 x NaN are NaN, for the query's heads that hold it and no others."""
    cache, table, lens, q = one(length, dtype)
    want = A.attention_step(q, cache, table, lens, scale=0.0)
    q[0, 2, 7] = value
    o = A.attention_step(q, cache, table, lens, scale=0.0)
    assert torch.isnan(o[0, 2]).all()
    o[0, 2] = want[0, 2]
    assert torch.equal(o, want)

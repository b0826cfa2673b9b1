"""Attention over prompts where q, k, v or dy hold something that is not finite and is seen: each
result is of the formula's class (not_finite_reference.agree)."""
from __future__ import annotations

import math

import pytest
import torch

import not_finite_reference as N
from attention_reference import half_step, seen
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


def prompt(dtype, lq=90, lk=150, hq=2, hk=1, dh=40):
    q, dy = rand((lq, hq, dh), 1, dtype, 2.0), rand((lq, hq, dh), 4, dtype)
    k, v = rand((lk, hk, dh), 2, dtype), rand((lk, hk, dh), 3, dtype)
    # channel 7 has one sign in all queries and keys: an infinite key or query there has scores
    # of one sign, in any other channel of both
    q[..., 7], k[..., 7] = q[..., 7].abs() + 0.5, k[..., 7].abs() + 0.5
    return q, k, v, dy


def hold(q, k, v, dy, scale, causal, window, dtype, skip=()):
    """The call's results against the formula's classes."""
    how = dict(scale=scale, causal=causal, window=window)
    o, lse = A.attention_forward(q, k, v, **how)
    grads = A.attention_backward(q, k, v, o, lse, dy, **how)
    ok = seen(q.shape[0], k.shape[0], causal, window, q.device)
    hq, hk = q.shape[1], k.shape[1]
    out = half_step(dtype) * 1.02
    sums = {x: [[0.0, 0.0] for _ in range(hk)] for x in ("dk", "dv")}
    for h in range(hq):
        g = h // (hq // hk)
        want, want_lse, bound, lse_bound = N.forward(q[:, h], k[:, g], v[:, g], ok, scale, dtype)
        N.agree(f"o, head {h}", o[:, h], want, bound)
        none = want_lse == -math.inf       # no key, or none with a score
        assert (torch.isnan(lse[h][none]) | (lse[h][none] == -math.inf)).all()
        N.agree(f"lse, head {h}", lse[h][~none], want_lse[~none], lse_bound[~none])
        got = N.backward(q[:, h], k[:, g], v[:, g], dy[:, h], o[:, h], lse[h], ok, scale, dtype)
        want, bound = got["dq"]
        N.agree(f"dq, head {h}", grads["dq"][:, h], want, bound * 1.05 + out * want.abs())
        for x in sums:
            sums[x][g][0], sums[x][g][1] = sums[x][g][0] + got[x][0], sums[x][g][1] + got[x][1]
    for x in sums:
        for g, (want, bound) in enumerate(sums[x]):
            N.agree(f"{x}, key head {g}", grads[x][:, g], want, bound * 1.05 + out * want.abs())


MASKS = [(True, 0), (True, 30), (False, 0)]


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("channel", [5, 7, None])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["k", "v"])
def test_class_of_results_keys(what, dtype, channel, value):
    """One channel of a key or value, or all of them, at the 100th of 150."""
    for scale in (40 ** -0.5, -0.5):
        for causal, window in MASKS:
            q, k, v, dy = prompt(dtype)
            t = k if what == "k" else v
            t[100, 0, slice(None) if channel is None else channel] = value
            hold(q, k, v, dy, scale, causal, window, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [40, 64, 96, 128])
def test_a_key_of_minus_infinity(dh, dtype):
    """A key whose score is minus infinity has no weight: every result but dq in the channel that
    is not finite is bit for bit that of a key with a score so low that its weight is zero."""
    n = 700
    q, k, v, dy = prompt(dtype, n, n, 4, 2, dh)
    for low in (-1e30, -math.inf):
        k[300, 1, 7] = low
        o, lse = A.attention_forward(q, k, v)
        got = [o, lse, *A.attention_backward(q, k, v, o, lse, dy).values()]
        if low == -1e30:
            want = got
    dq = got[2]
    assert torch.isnan(dq[300:, 2:, 7]).all()
    dq[300:, 2:, 7] = want[2][300:, 2:, 7]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("channel", [5, 7, None])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["q", "dy"])
def test_class_of_results_queries(what, dtype, channel, value):
    """The same of a query and its gradient, at the 50th of 90."""
    for scale in (40 ** -0.5, -0.5):
        for causal, window in MASKS:
            q, k, v, dy = prompt(dtype)
            t = q if what == "q" else dy
            t[50, 1, slice(None) if channel is None else channel] = value
            hold(q, k, v, dy, scale, causal, window, dtype)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_scale_of_zero(what, dtype, value):
    """0 x infinity and 0 x NaN are NaN."""
    q, k, v, dy = prompt(dtype)
    if what == "q":
        q[50, 1, 5] = value
    else:
        k[100, 0, 5] = value
    hold(q, k, v, dy, 0.0, True, 0, dtype)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [72, 128])
def test_class_of_results_shared_tiles(dh, dtype, value):
    """Groups of four heads, where blocks share a tile of keys and leave partial sums."""
    for what in range(4):
        t = prompt(dtype, 300, 300, 4, 1, dh)
        t[what][170, 0, 7] = value
        hold(*t, dh ** -0.5, True, 0, dtype)

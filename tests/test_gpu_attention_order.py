"""Attention over prompts whose tiles are sorted by their work: batches of several sequences with
more tiles than run at once (over 512, of all heads), to 1024 sequences and 2048 tiles.

A batch's results are those of its sequences alone, whose tiles are not sorted: o, lse and dq to the
bit (a sequence's tiles begin with it); dk and dv, whose sums the blocks share otherwise in small
calls, within the bounds of the 64-bit form."""
from __future__ import annotations

import math

import pytest
import torch

import attention_reference as R
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
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)


def inputs(lq, lk, hq, hk, dh, dtype, tail=0):
    n, nk = sum(lq) + tail, sum(lk) + tail
    return (rand((n, hq, dh), 1, dtype, 2.0), rand((nk, hk, dh), 2, dtype), rand((nk, hk, dh), 3, dtype),
            rand((n, hq, dh), 4, dtype))


def sorted_tiles(lq, lk, hq, hk, tail=0):
    for lens, heads in ((lq, hq), (lk, hk)):
        tiles = (sum(lens) + tail) // 128 + len(lens) + 1
        assert 1 < len(lens) <= 1024 and tiles <= 2048 and tiles * heads > 512


LENS = [700, 0, 1, 1300, 999]
CASES = [  # lens of queries, of keys, causal, window, rows behind the last sequence
    (LENS, LENS, True, 0, 0),
    (LENS, LENS, True, 0, 200),
    (LENS, LENS, True, 100, 0),
    (LENS, [1000, 0, 6, 1364, 1999], True, 0, 0),          # keys from before
    (LENS, [1000, 0, 6, 1364, 1999], True, 900, 31),
    (LENS, [300, 5, 0, 1300, 2500], True, 0, 0),           # queries that see no key
    (LENS, [300, 5, 0, 1300, 2500], True, 1200, 0),
    (LENS, [300, 5, 0, 1300, 2500], False, 0, 77),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES)
def test_sorted_tiles(case, dtype):
    lq, lk, causal, window, tail = case
    hq = hk = 32
    sorted_tiles(lq, lk, hq, hk, tail)
    q, k, v, dy = inputs(lq, lk, hq, hk, 16, dtype, tail)
    how = dict(causal=causal, window=window)
    at = dict(offsets=offsets(lq), k_offsets=offsets(lk))
    o, lse = A.attention_forward(q, k, v, **at, **how)
    got = A.attention_backward(q, k, v, o, lse, dy, **at, **how)
    for rows, keys in R.sequences(lq, lk):
        alone = q[rows], k[keys], v[keys]
        oo, ll = A.attention_forward(*alone, **how)
        assert torch.equal(o[rows], oo) and torch.equal(lse[:, rows], ll)
        if rows.stop > rows.start:
            dq = A.attention_backward(*alone, oo, ll.contiguous(), dy[rows], **how)["dq"]
            assert torch.equal(got["dq"][rows], dq)
    m, mk = sum(lq), sum(lk)
    assert (o[m:] == 0).all() and (lse[:, m:] == -math.inf).all() and (got["dq"][m:] == 0).all()
    assert (got["dk"][mk:] == 0).all() and (got["dv"][mk:] == 0).all()
    want, bound = R.attention_backward(q, k, v, o, lse, dy, lq, lk, causal, window)
    for x in ("dq", "dk", "dv"):
        assert ((got[x].double() - want[x]).abs() <= bound[x]).all(), x


@pytest.mark.parametrize("batch", [1024, 1025])
def test_either_side_of_the_most_sequences(batch):
    lens = [(i * 7) % 5 for i in range(batch)]
    q, k, v, dy = inputs(lens, lens, 2, 1, 16, BF16)
    at = dict(offsets=offsets(lens))
    o, lse = A.attention_forward(q, k, v, **at)
    want, want_lse, bound, lse_bound = R.attention(q, k, v, lens, lens)
    assert ((o.double() - want).abs() <= bound).all() and ((lse.double() - want_lse).abs() <= lse_bound).all()
    got = A.attention_backward(q, k, v, o, lse, dy, **at)
    want, bound = R.attention_backward(q, k, v, o, lse, dy, lens, lens)
    for x in want:
        assert ((got[x].double() - want[x]).abs() <= bound[x]).all(), x


@pytest.mark.parametrize("tiles", [2048, 2049])
def test_either_side_of_the_most_tiles(tiles):
    """Two long sequences with a short window against the two alone: all bit for bit, since tiles
    of so many keys are not shared."""
    n = (tiles - 3) * 128
    lens = [200_001, n - 200_001]
    q, k, v, dy = inputs(lens, lens, 1, 1, 8, BF16)
    o, lse = A.attention_forward(q, k, v, offsets=offsets(lens), window=60)
    got = A.attention_backward(q, k, v, o, lse, dy, offsets=offsets(lens), window=60)
    for rows, _ in R.sequences(lens, lens):
        alone = q[rows], k[rows], v[rows]
        oo, ll = A.attention_forward(*alone, window=60)
        assert torch.equal(o[rows], oo) and torch.equal(lse[:, rows], ll)
        want = A.attention_backward(*alone, oo, ll, dy[rows], window=60)
        assert all(torch.equal(got[x][rows], want[x]) for x in want)


def test_sorted_and_replayed():
    """A captured training step, replayed with other offsets: the order is made anew."""
    lens = [LENS, [0, 0, 2000, 900, 100], [2990, 1, 3, 3, 3], [5, 5, 5, 5, 5]]
    q, k, v, dy = inputs(LENS, LENS, 32, 32, 16, BF16)
    off = offsets(LENS)

    def step():
        o, lse = A.attention_forward(q, k, v, offsets=off)
        return [o, lse, *A.attention_backward(q, k, v, o, lse, dy, offsets=off).values()]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for m in lens[1:] + lens[:1]:
        off.copy_(offsets(m))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        torch.cuda.synchronize()


def test_sorted_offsets_that_fall():
    """Falling offsets stay within the tensors."""
    n = 3000
    q, k, v, dy = inputs([n], [n], 32, 32, 16, BF16)
    for off in ([0, 40, 20, -5, 7, 2900], [5, 4, 3, 2, 1, 0], [0, 2000, 1000, 3000, 0, 1], [9, -9, 10 ** 9, 0, 3000, 0]):
        off = torch.tensor(off, dtype=torch.int32, device=DEV)
        o, lse = A.attention_forward(q, k, v, offsets=off)
        A.attention_backward(q, k, v, o, lse, dy, offsets=off)
        torch.cuda.synchronize()

"""The attention operators on a stream other than the current one, captured into graphs and
replayed, two at once, and beyond 2^31 elements."""
from __future__ import annotations

import pytest
import torch

import attention_reference as R
from chunked_weight_mlp_amd import attention as A
from chunked_weight_mlp_amd.ipttt import IptttError

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
WAIT = 20_000_000   # ticks of the device's clock: milliseconds


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.load()


def rand(shape, seed, dtype=BF16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def inputs(dtype=BF16):
    """Everything the calls read."""
    n, hq, hk, dh, page = 500, 8, 2, 64, 16
    inv = 1e4 ** (-torch.arange(0, dh, 2, dtype=torch.float64) / dh).to(DEV)
    t = dict(q=rand((n, hq, dh), 1, dtype, 2.0), k=rand((n, hk, dh), 2, dtype), v=rand((n, hk, dh), 3, dtype),
             dy=rand((n, hq, dh), 4, dtype), dk=rand((n, hk, dh), 5, dtype),
             pos=torch.arange(n, dtype=torch.int32, device=DEV),
             off=torch.tensor([0, 130, 131, n], dtype=torch.int32, device=DEV),
             lens=torch.tensor([1600, 33], dtype=torch.int32, device=DEV),
             table=torch.randperm(240, generator=torch.Generator().manual_seed(6)).to(torch.int32).view(2, 120).to(DEV),
             at=torch.tensor([1599, 32], dtype=torch.int32, device=DEV))
    t["op"] = A.HeadNorm(rand((dh,), 7, dtype), rand((dh,), 8, dtype), inv)
    t["cache"] = A.KVCache(rand((240, hk, page, dh), 9, dtype), rand((240, hk, page, dh), 10, dtype))
    t["o"], t["lse"] = A.attention_forward(t["q"], t["k"], t["v"], offsets=t["off"])
    return t


CALLS = {
    "heads forward": lambda t, st: t["op"].forward(t["q"], t["k"], t["pos"], stream=st),
    "heads append": lambda t, st: t["op"].append(t["q"][:2], t["k"][:2], t["v"][:2], t["at"], t["cache"], t["table"],
                                                 stream=st),
    "heads backward": lambda t, st: t["op"].backward(t["q"], t["k"], t["pos"], t["dy"], t["dk"], stream=st),
    "attention forward": lambda t, st: A.attention_forward(t["q"], t["k"], t["v"], offsets=t["off"], stream=st),
    "attention backward": lambda t, st: A.attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["dy"],
                                                             offsets=t["off"], stream=st),
    "attention step": lambda t, st: A.attention_step(t["q"][:2], t["cache"], t["table"], t["lens"], stream=st),
}


def results(out):
    return [out] if isinstance(out, torch.Tensor) else list(out.values()) if isinstance(out, dict) else list(out)


def same(got, want):
    assert len(got) == len(want)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_memory_the_current_stream_still_writes(name, handle):
    """Late writes of the current stream to tensors that are gone when the call is made, of
    every size from small ones to the call's largest."""
    t = inputs()
    want = [x.clone() for x in results(CALLS[name](t, None))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    gone = [torch.empty(1 << k, dtype=torch.uint8, device=DEV) for k in range(9, 23) for _ in range(4)]
    gone += [torch.empty_like(x) for x in want for _ in range(2)]
    torch.cuda._sleep(WAIT)
    for x in gone:
        x.view(torch.uint8).fill_(0xff)
    del gone, x
    out = results(CALLS[name](t, s.cuda_stream if handle else s))
    torch.cuda.synchronize()
    same(out, want)


@pytest.mark.parametrize("name", CALLS)
def test_memory_the_other_stream_still_uses(name):
    """Writes of the current stream, made at once, while the call waits on its stream: to
    whatever the call has given back, its workspace among it; and to inputs given back."""
    t = inputs()
    want = [x.clone() for x in results(CALLS[name](t, None))]
    if name == "heads append":
        t = inputs()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    out = results(CALLS[name](t, s))
    del t
    for k in range(9, 25):
        for _ in range(4):
            torch.empty(1 << k, dtype=torch.uint8, device=DEV).fill_(0xff)
    for x in want:
        torch.empty_like(x).view(torch.uint8).fill_(0xff)
    torch.cuda.synchronize()
    same(out, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(name, dtype):
    """A graph of the call, replayed with other inputs in the same tensors and eager work and
    synchronisations between, gives what the eager call gives."""
    t = inputs(dtype)
    CALLS[name](t, None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = results(CALLS[name](t, None))
    for k in range(3):
        for i, x in enumerate(("q", "k", "v", "dy", "dk")):
            t[x].copy_(rand(t[x].shape, 100 + 10 * k + i, dtype))
        t["lens"].copy_(torch.tensor([[1600, 33], [7, 1900], [0, 480]][k], dtype=torch.int32))
        t["off"].copy_(torch.tensor([[0, 130, 131, 500], [0, 0, 250, 400], [0, 500, 500, 500]][k], dtype=torch.int32))
        if name == "attention backward":
            o, lse = A.attention_forward(t["q"], t["k"], t["v"], offsets=t["off"])
            t["o"].copy_(o), t["lse"].copy_(lse)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        same(got, results(CALLS[name](t, None)))
        torch.cuda.synchronize()


def test_two_graphs_replayed_in_turn():
    """Graphs of a decode step and of a training step, whose workspaces come from one pool."""
    t = inputs()
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for name in ("attention step", "attention backward"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(results(CALLS[name](t, None)))
        pool = pool or g.pool()
        graphs.append(g)
    want = [[x.clone() for x in results(CALLS[n](t, None))] for n in ("attention step", "attention backward")]
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        same(outs[0], want[0])
        same(outs[1], want[1])


def test_two_calls_at_once():
    t = inputs()
    want = {n: [x.clone() for x in results(CALLS[n](t, None))] for n in CALLS if n != "heads append"}
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(n, results(CALLS[n](t, streams[i % 3]))) for i, n in enumerate(want)]
        torch.cuda.synchronize()
        for n, out in got:
            same(out, want[n])


def test_autograd_is_left_alone():
    """Inputs that require a gradient are used by their value."""
    t = inputs()
    q = t["q"].clone().requires_grad_()
    o, lse = A.attention_forward(q, t["k"], t["v"], offsets=t["off"])
    assert not o.requires_grad and torch.equal(o, t["o"])
    assert not t["op"].forward(q, t["k"], t["pos"])[0].requires_grad


def test_beyond_31_bits():
    """A cache and heads whose elements are further than 2^31 from their first one."""
    hk, page, dh = 8, 64, 128
    pages = (2 ** 31) // (hk * page * dh) + 40
    k, v = (torch.zeros((pages, hk, page, dh), dtype=BF16, device=DEV) for _ in range(2))
    n = 1000
    mine = torch.tensor([pages - 1 - 2 * i for i in range(-(-n // page))], dtype=torch.int32)
    for t, s in ((k, 1), (v, 2)):
        t[mine.long().to(DEV)] = rand((len(mine), hk, page, dh), s)
    cache, table = A.KVCache(k, v), mine[None].to(DEV)
    q, lens = rand((1, 16, dh), 3, BF16, 2.0), torch.tensor([n], dtype=torch.int32, device=DEV)
    want, bound = R.step(q, k, v, table, lens)
    o = A.attention_step(q, cache, table, lens)
    assert ((o.double() - want).abs() <= bound).all()
    inv = 1e4 ** (-torch.arange(0, dh, 2, dtype=torch.float64) / dh).to(DEV)
    op = A.HeadNorm(rand((dh,), 4), rand((dh,), 5), inv)
    new = rand((1, 32, dh), 6)
    pos = torch.tensor([n], dtype=torch.int32, device=DEV)
    op.append(new[:, :16], new[:, 16:24], new[:, 24:], pos, cache, table)
    at = int(mine[n // page])
    assert torch.equal(v[at, :, n % page], new[0, 24:])
    assert torch.equal(k[at, :, n % page], op.forward(new[:, :16], new[:, 16:24], pos)[1][0])
    del k, v, cache
    # tokens 2^25 elements apart
    m, wide = 70, 1 << 25
    buf = torch.empty((m, wide), dtype=BF16, device=DEV)
    q = buf[:, wide - 3 * dh:wide - dh].view(m, 2, dh)
    kk = buf[:, :dh].view(m, 1, dh)
    q.copy_(rand((m, 2, dh), 7, BF16, 2.0)), kk.copy_(rand((m, 1, dh), 8))
    dense = [x.contiguous() for x in (q, kk)]
    o, lse = A.attention_forward(q, kk, kk)
    same([o, lse], A.attention_forward(dense[0], dense[1], dense[1]))
    dy = rand((m, 2, dh), 9)
    same(results(A.attention_backward(q, kk, kk, o, lse, dy)),
         results(A.attention_backward(dense[0], dense[1], dense[1], o, lse, dy)))
    pos = torch.arange(m, dtype=torch.int32, device=DEV)
    same(op.forward(q, kk, pos), op.forward(*dense, pos))


def test_another_device_is_refused():
    t = inputs()
    with pytest.raises(IptttError):
        A.attention_forward(t["q"], t["k"].cpu(), t["v"], offsets=t["off"])
    with pytest.raises(IptttError):
        A.attention_step(t["q"][:2], t["cache"], t["table"].cpu(), t["lens"])
    with pytest.raises(IptttError):
        t["op"].forward(t["q"], t["k"], t["pos"].cpu())

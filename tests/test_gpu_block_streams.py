"""The block operators on a stream other than the current one (`stream=`): memory that
one of the two streams still works on is not handed to the other.

Each test queues a wait on one stream and, behind it, writes to memory that has been
given back to the allocator by then. Sizes are those of the call's own workspace and
outputs, so that an allocation that could be handed such a block is handed it: what is
written late then shows in the results."""
from __future__ import annotations

import pytest
import torch

from chunked_weight_mlp_amd import block as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
WAIT = 20_000_000   # ticks of the device's clock: milliseconds


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.load()


def rand(shape, seed, dtype=F32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)


def calls():
    """name -> (call(stream), its workspace in bytes)."""
    n, d, f, length = 300, 192, 320, 2000
    norm = K.Norm(rand((d,), 1, BF16, 0.2, 1.0), rand((d,), 2, BF16))
    x, r, dy = rand((n, d), 3, BF16), rand((n, d), 4, BF16), rand((n, d), 5, BF16)
    _, h, mean, rstd = norm.forward(x, r)
    ff = K.FeedForward(rand((f, d), 6, BF16, d ** -0.5), rand((f, d), 7, BF16, d ** -0.5),
                       rand((d, f), 8, BF16, f ** -0.5))
    _, a, u = ff.forward(x, save=True)
    g, v, dh = (rand((2, length, d), k, BF16, 2.0, m) for k, m in ((9, 2.0), (10, 0.0), (11, 0.0)))
    s, _ = K.recurrence_forward(g, v)
    state = rand((2, d), 12)
    rec = K.ipttt_recurrence_workspace_bytes(K._recurrence(g, v, s, None))
    return {
        "norm forward": (lambda st: norm.forward(x, r, stream=st), 0),
        "norm backward": (lambda st: norm.backward(h, mean, rstd, dy, r, stream=st),
                          K.ipttt_norm_backward_workspace_bytes(norm.desc, n)),
        "recurrence forward": (lambda st: K.recurrence_forward(g, v, stream=st), rec),
        "recurrence step": (lambda st: K.recurrence_step(g[:, 0], v[:, 0], state, stream=st), 0),
        "recurrence backward": (lambda st: K.recurrence_backward(g, v, s, dh, stream=st), rec),
        "ff forward": (lambda st: ff.forward(x, save=True, stream=st), K.ipttt_ff_workspace_bytes(ff.desc, n)),
        "ff backward": (lambda st: ff.backward(x, a, u, dy, stream=st),
                        K.ipttt_ff_backward_workspace_bytes(ff.desc, n)),
    }


CALLS = ("norm forward", "norm backward", "recurrence forward", "recurrence step",
         "recurrence backward", "ff forward", "ff backward")


def results(out):
    return list(out.values()) if isinstance(out, dict) else list(out)


def blocks(out, ws):
    """Two tensors of every size the call allocates."""
    sizes = [t.numel() * t.element_size() for t in results(out)] + ([ws] if ws else [])
    return [torch.empty(b, dtype=torch.uint8, device=DEV) for b in sizes for _ in range(2)]


def same(got, want):
    assert len(got) == len(want)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_memory_the_current_stream_still_writes(name, handle):
    """Late writes of the current stream to tensors that are gone when the call is made."""
    call, ws = calls()[name]
    want = [t.clone() for t in results(call(None))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    gone = blocks(want, ws)
    torch.cuda._sleep(WAIT)
    for t in gone:
        t.fill_(0xff)
    at = {t.data_ptr() for t in gone}
    del gone, t
    out = results(call(s.cuda_stream if handle else s))
    assert not at & {t.data_ptr() for t in out}
    torch.cuda.synchronize()
    same(out, want)


@pytest.mark.parametrize("name", CALLS)
def test_memory_the_other_stream_still_uses(name):
    """Writes of the current stream, made at once, while the call waits on its stream:
    to whatever the call has given back, which is its workspace."""
    call, ws = calls()[name]
    want = [t.clone() for t in results(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    out = results(call(s))
    for t in blocks(want, ws):
        t.fill_(0xff)
    torch.cuda.synchronize()
    same(out, want)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_the_current_stream_still_reads(name):
    """Outputs read late on the current stream and given back before that: the other
    stream's next allocations do not get them."""
    call, ws = calls()[name]
    want = [t.clone() for t in results(call(None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = results(call(s))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(WAIT)
    kept = [t.clone() for t in out]
    del out
    with torch.cuda.stream(s):
        for t in blocks(want, ws):
            t.fill_(0xff)
    torch.cuda.synchronize()
    same(kept, want)


@pytest.mark.parametrize("name", CALLS)
def test_inputs_given_back_before_the_call_has_run(name):
    """Inputs whose last reference goes while the call waits: their memory is not reused."""
    made = calls()
    call, ws = made[name]
    want = [t.clone() for t in results(call(None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    out = results(call(s))
    sizes = {c.cell_contents.numel() * c.cell_contents.element_size()
             for c in call.__closure__ if isinstance(c.cell_contents, torch.Tensor)}
    del made, call
    for b in sizes:
        for _ in range(4):
            torch.empty(b, dtype=torch.uint8, device=DEV).fill_(0xff)
    torch.cuda.synchronize()
    same(out, want)


def test_the_current_stream_given_as_stream():
    call, _ = calls()["ff forward"]
    same(results(call(torch.cuda.current_stream())), results(call(None)))

"""The gated linear recurrence with gates that remember (f near 1): what a tile of
tokens hands to the tiles behind it is most of their state, over groups of tiles and
past the window of groups a tile looks at, both ways, and a state is kept as long as the
formula says.

Tolerances, fixed from the arithmetic. fp32 state and gradient: e^-g is off by |g| 2^-24
of itself (g up to 12: 7e-7), which moves a result by at most that times k (1 - f) f^k <=
0.37; a result passes about ten roundings of 2^-24 in its tile and one per group of tiles
before it, whose sizes fall off like the state itself, adding in quadrature, and rounded
factors of up to 16 tokens, 16 x 2^-25: 1e-6 in all, 5e-6 allowed (rounded factors f alone would leave 3e-5, 5e-4 and 7e-3 at g = 8, 10 and 12).
dg adds the difference h - v and three products: the same bound. Handed on in fp32 from call to call, a state is rounded at every call: sqrt(2^17)
2^-25 = 1.1e-5 over 2^17 roundings that are independent, 4e-5 allowed for calls of 16
tokens and more (rounded at every token, those of one gate are not: 5e-4 at g = 14). bf16 results add one rounding, 4e-3."""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from chunked_weight_mlp_amd import block as K
from parity_check import rel_fro, report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 4e-3, "f32": 5e-6}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.load()


def rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


def close(got, want, tol, label):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), label
    e = rel_fro(got.numpy(), want.numpy())
    report(f"[recurrence, remembering] {label}: rel_fro {e:.2e} (tol {tol:.0e})")
    assert e <= tol, (label, e)


def remembering(n, length, d, t, mean, starts, lens):
    """Gates about `mean`, a state before and a gradient behind that are larger than the
    values, document starts at the given (sequence, token) places."""
    g, v = rand((n, length, d), 1, t, 0.3, mean), rand((n, length, d), 2, t)
    st = ln = None
    if starts is not None:
        st = torch.zeros((n, length), dtype=torch.uint8)
        for i, at in starts:
            st[i, at] = 1
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int32)
        for i, m in enumerate(lens):
            g[i, m:], v[i, m:] = float("nan"), float("nan")
    return g, v, rand((n, d), 3, std=3.0), st, ln


# 40 to 80 tiles of 128 tokens: 5 to 10 groups of 8 tiles, of which a tile sees 8
MEMORY = [
    (1, 10241, 3, 8.0, None, None),
    (2, 5120, 65, 7.0, None, None),
    (3, 3001, 130, 9.0, [(1, 1500), (2, 300), (2, 2999)], None),
    (3, 6000, 33, 8.0, [(1, 0), (2, 4095), (2, 4096)], [6000, 2561, 4224]),
    (4, 2700, 64, 7.0, None, [2700, 1, 129, 2048]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,length,d,mean,starts,lens", MEMORY)
def test_state_carried_over_tiles(dtype, n, length, d, mean, starts, lens):
    t = TYPES[dtype]
    g, v, h0, st, ln = remembering(n, length, d, t, mean, starts, lens)
    tag = f"{dtype} {n}x{length}x{d}"
    h, last = K.recurrence_forward(dev(g), dev(v), h0=dev(h0), starts=dev(st), lens=dev(ln))
    want, wlast = ref.recurrence(g, v, h0, st, ln)
    close(h, want, TOL[dtype], tag + " h")
    close(last, wlast, 5e-6, tag + " last")
    # the state before counts: a tile keeps most of what it is given
    forgot = ref.recurrence(g[:, :256], v[:, :256], torch.zeros_like(h0), None, None)[0]
    assert rel_fro(forgot[0, 255].numpy(), want[0, 255].numpy()) > 0.3
    dh, dl = rand((n, length, d), 4, t, 0.1), rand((n, d), 5, std=3.0)
    if lens is not None:
        for i, m in enumerate(lens):
            dh[i, m:] = float("nan")
    got = K.recurrence_backward(dev(g), dev(v), h, dev(dh), h0=dev(h0), dh_last=dev(dl), starts=dev(st),
                                lens=dev(ln))
    dg, dv, dh0 = ref.recurrence_backward(g, v, h.cpu(), dh, h0, dl, st, ln)
    close(got["dg"], dg, TOL[dtype], tag + " dg")
    close(got["dv"], dv, TOL[dtype], tag + " dv")
    close(got["dh0"], dh0, 5e-6, tag + " dh0")


def vector_reference(g, v, h0, dh, dl):
    """One sequence [length, d] both ways in 64 bits."""
    g, v, dh, s = g.double(), v.double(), dh.double(), h0.double()
    f, i = torch.sigmoid(g), torch.sigmoid(-g)
    h = torch.empty_like(g)
    for t in range(len(g)):
        s = torch.addcmul(i[t] * v[t], f[t], s, out=h[t])
    delta, s = torch.empty_like(g), dl.double()
    for t in range(len(g) - 1, -1, -1):
        torch.add(dh[t], s, out=delta[t])
        s = f[t] * delta[t]
    prev = torch.cat([h0.double()[None], h[:-1]])
    return h, delta * (prev - v) * f * i, i * delta, s


GATES = (6.0, 8.0, 10.0, 12.0, 14.0)


def constant_gates(length, each, dtype):
    """Channels of one gate each, `each` of every value in GATES."""
    d = each * len(GATES)
    g = torch.tensor(GATES).repeat_interleave(each).expand(length, d).contiguous()
    return (g.to(dtype), rand((length, d), 1, dtype, 0.01), rand((d,), 2).abs() + 1,
            rand((length, d), 3, dtype, 0.01), rand((d,), 4).abs() + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_constant_gates_over_a_long_sequence(dtype):
    """131072 tokens of one gate a channel: a bias of f would add up over all of them."""
    each = 16
    g, v, h0, dh, dl = constant_gates(131072, each, TYPES[dtype])
    want, dg, dv, dh0 = vector_reference(g, v, h0, dh, dl)
    h, last = K.recurrence_forward(dev(g)[None], dev(v)[None], h0=dev(h0)[None])
    got = K.recurrence_backward(dev(g)[None], dev(v)[None], want.to(TYPES[dtype])[None].to(DEV),
                                dev(dh)[None], h0=dev(h0)[None], dh_last=dev(dl)[None])
    for k, gate in enumerate(GATES):
        c = slice(k * each, (k + 1) * each)
        tag = f"{dtype} 131072 tokens, g = {gate:.0f}"
        close(h[0, :, c], want[:, c], TOL[dtype], tag + " h")
        close(last[0, c], want[-1, c], 5e-6, tag + " last")
        close(got["dv"][0, :, c], dv[:, c], TOL[dtype], tag + " dv")
        close(got["dh0"][0, c], dh0[c], 5e-6, tag + " dh0")
        close(got["dg"][0, :, c], dg[:, c], TOL[dtype] if dtype == "f32" else 8e-3, tag + " dg")


@pytest.mark.parametrize("call", [16, 100, 1000])
def test_constant_gates_in_short_calls(call):
    """The same in many calls, the state handed on: walked token by token, in one tile, in
    several."""
    each, length = 8, 1 << 17
    g, v, h0, dh, dl = constant_gates(length, each, torch.float32)
    want, _, _, dh0 = vector_reference(g, v, h0, dh, dl)
    gd, vd, hd, dhd = dev(g)[None], dev(v)[None], want.float()[None].to(DEV), dev(dh)[None]
    s = dev(h0)[None]
    for at in range(0, length, call):
        _, s = K.recurrence_forward(gd[:, at:at + call], vd[:, at:at + call], h0=s)
    G = dev(dl)[None]
    for at in reversed(range(0, length, call)):
        part = slice(at, at + call)
        G = K.recurrence_backward(gd[:, part], vd[:, part], hd[:, part], dhd[:, part], dh_last=G)["dh0"]
    for k, gate in enumerate(GATES):
        c = slice(k * each, (k + 1) * each)
        close(s[0, c], want[-1, c], 4e-5, f"calls of {call}, g = {gate:.0f} last")
        close(G[0, c], dh0[c], 4e-5, f"calls of {call}, g = {gate:.0f} dh0")


def test_infinite_states_stay_infinite():
    """A state or a gradient that is infinite is not made NaN by a gate that keeps it, in
    tiles and walked; one that a document start cuts is gone."""
    for length in (9, 700):
        g = rand((1, length, 6), 1, std=0.5, mean=9.0)
        g[0, 5] = -1.0
        v = rand((1, length, 6), 2)
        h0 = torch.zeros(1, 6)
        h0[0, 1], h0[0, 4] = float("inf"), -float("inf")
        st = torch.zeros((1, length), dtype=torch.uint8)
        h, last = K.recurrence_forward(dev(g), dev(v), h0=dev(h0))
        want, wlast = ref.recurrence(g, v, h0, None, None)
        assert torch.isposinf(h[0, :, 1]).all() and torch.isneginf(h[0, :, 4]).all()
        ok = [0, 2, 3, 5]
        assert rel_fro(h[..., ok].cpu().numpy(), want[..., ok].numpy()) <= 5e-6
        assert torch.equal(torch.isinf(last.cpu()), torch.isinf(wlast))
        st[0, length - 3] = 1
        h, last = K.recurrence_forward(dev(g), dev(v), h0=dev(h0), starts=dev(st))
        assert torch.isfinite(h[0, length - 3:]).all() and torch.isfinite(last).all()
        dl = h0
        got = K.recurrence_backward(dev(g), dev(v), dev(want.float().nan_to_num(0, 0, 0)), dev(v), dh_last=dev(dl))
        assert torch.isposinf(got["dv"][0, :, 1]).all() and torch.isneginf(got["dv"][0, :, 4]).all()
        assert torch.equal(torch.isinf(got["dh0"].cpu()), torch.isinf(dl))


@pytest.mark.parametrize("n,length,d", [(2, 6000, 300), (1, 60001, 43), (9, 3000, 517)])
def test_remembering_repeats_bit_for_bit(n, length, d):
    """Whole states pass through the chain, so an order that depended on timing would show."""
    g, v, h0, _, _ = remembering(n, length, d, torch.float32, 8.0, None, None)
    g, v, h0 = dev(g), dev(v), dev(h0)
    first = K.recurrence_forward(g, v, h0=h0)
    grads = K.recurrence_backward(g, v, first[0], v, h0=h0, dh_last=h0)
    for _ in range(4):
        again = K.recurrence_forward(g, v, h0=h0)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        for k, t in K.recurrence_backward(g, v, again[0], v, h0=h0, dh_last=h0).items():
            assert torch.equal(grads[k], t), k

"""The block operators (include/ipttt_block.h) on the GPU against their formulas in
64 bits: sizes from one token up, odd widths, strided inputs, cut and ragged
sequences, non-finite padding, and the gradients against differences.

Tolerances (relative Frobenius error unless an entry says otherwise), fixed from
the arithmetic. A value rounded to bf16 once is off by at most 2^-8 of itself,
3.9e-3, and 1.7e-3 in the mean square: 4e-3 for one rounding. A feed-forward
output passes through up to four such roundings (a, u, z or dA, the output),
3.4e-3 in the mean square over many values and 1.6e-2 at worst in one value:
8e-3 for results of 64 values or more, 2e-2 for smaller ones. fp32 results carry a few 2^-24 roundings and the hardware
exponential's error (|x| 2^-24 for e^x, |x| < 20 here): 5e-6, and 2e-5 where
the recurrence and its gradient chain many of them.
"""
from __future__ import annotations

import pytest
import torch

import block_reference as ref
from chunked_weight_mlp_amd import block as K
from chunked_weight_mlp_amd import ipttt as B
from parity_check import rel_fro, report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ONE = {"bf16": 4e-3, "f32": 5e-6}       # one rounding of the type
CHAIN = {"bf16": 4e-3, "f32": 2e-5}     # recurrence
FF = {"bf16": 8e-3, "f32": 2e-5}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.load()


def rand(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def wide(t, pad):
    """The same values on the GPU as a slice of rows that are `pad` elements longer."""
    if not pad:
        return t.to(DEV)
    w = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=DEV)
    w[..., : t.shape[-1]] = t.to(DEV)
    return w[..., : t.shape[-1]]


def close(got, want, tol, label):
    got = got.double().cpu()
    assert got.shape == want.shape, (label, got.shape, want.shape)
    assert torch.isfinite(got).all(), label
    if want.numel() == 0:
        return
    if float(want.norm()) == 0.0:
        assert float(got.abs().max()) == 0.0, label
        return
    e = rel_fro(got.numpy(), want.numpy())
    report(f"[block] {label}: rel_fro {e:.2e} (tol {tol:.0e})")
    assert e <= tol, (label, e)


# ---- layer norm -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,pad", [
    (1, 1, 0), (3, 7, 0), (5, 64, 3), (2, 513, 0), (9, 1024, 8), (4, 1543, 1), (2100, 1030, 0),
    (3, 2560, 0), (2050, 2560, 0), (2, 4097, 0), (3, 8192, 8), (2, 16384, 0), (1, 16383, 5)])
def test_norm(dtype, n, d, pad):
    t = TYPES[dtype]
    x, r = rand((n, d), 1, t, 3.0, 0.5), rand((n, d), 2, t)
    gamma, beta = rand((d,), 3, t, 0.2, 1.0), rand((d,), 4, t)
    op = K.Norm(gamma.to(DEV), beta.to(DEV), eps=1e-3)
    for res in (r, None):
        y, h, mean, rstd = op.forward(wide(x, pad), None if res is None else wide(res, 2 * pad))
        want = ref.norm_forward(x, res, gamma, beta, 1e-3)
        tag = f"norm {dtype} {n}x{d} pad {pad} {'add' if res is not None else ''}"
        close(y, want[0], ONE[dtype], tag + " y")
        close(h, want[1], ONE[dtype], tag + " h")
        close(mean, want[2], 5e-6, tag + " mean")
        close(rstd, want[3], 5e-6, tag + " rstd")
    dy, dh = rand((n, d), 5, t), rand((n, d), 6, t)
    for upstream in (dh, None):
        got = op.backward(h, mean, rstd, wide(dy, pad), None if upstream is None else wide(upstream, pad))
        dx, dgamma, dbeta = ref.norm_backward(x, mean.cpu(), rstd.cpu(), gamma, dy, upstream)
        tag = f"norm backward {dtype} {n}x{d} {'dh' if upstream is not None else ''}"
        if d > 1:   # with one column dx is dh alone, whose value the sum cancels to
            close(got["dx"], dx, ONE[dtype], tag + " dx")
            close(got["dgamma"], dgamma, 2e-5, tag + " dgamma")
        close(got["dbeta"], dbeta, 5e-6, tag + " dbeta")


def test_norm_without_weights_and_constant_rows():
    """gamma and beta NULL; a row of equal values has zero deviations: y = beta."""
    x = rand((6, 100), 1, std=2.0)
    x[2] = 5.0
    y = torch.empty((6, 100), device=DEV)
    desc = K.NormDesc(d=100, dtype=B.IPTTT_F32, eps=1e-5, gamma=None, beta=None)
    K.ipttt_norm_forward(desc, x.to(DEV), 100, None, 0, 6, None, y, None, None)
    close(y, ref.norm_forward(x, None, None, None, 1e-5)[0], 5e-6, "norm without weights")
    assert float(y[2].abs().max()) == 0.0


def test_norm_large_mean():
    """Deviations of 1 on a mean of 4096: the two-pass variance keeps them."""
    x = rand((8, 2048), 1, std=1.0, mean=4096.0)
    op = K.Norm(torch.ones(2048, device=DEV), None)
    y, _, _, rstd = op.forward(x.to(DEV))
    want = ref.norm_forward(x, None, None, None, 1e-5)
    close(rstd, want[3], 5e-6, "norm large mean rstd")
    # the mean itself is rounded to 2^-24 of 4096: 1.2e-4 of a deviation
    close(y, want[0], 5e-4, "norm large mean y")


def test_norm_no_rows():
    op = K.Norm(torch.ones(64, device=DEV), torch.zeros(64, device=DEV))
    e = torch.empty((0, 64), device=DEV)
    y, _, mean, rstd = op.forward(e)
    assert y.shape == (0, 64)
    got = op.backward(e, mean, rstd, e)
    torch.cuda.synchronize()
    assert float(got["dgamma"].abs().max()) == 0.0 and float(got["dbeta"].abs().max()) == 0.0


def test_norm_gradient_against_differences():
    """d(loss)/dx by central differences of the forward in 64 bits around the kernel's dx."""
    x, gamma, beta = rand((3, 33), 1, std=2.0), rand((33,), 2, mean=1.0), rand((33,), 3)
    dy = rand((3, 33), 4)
    op = K.Norm(gamma.to(DEV), beta.to(DEV))
    y, h, mean, rstd = op.forward(x.to(DEV))
    got = op.backward(h, mean, rstd, dy.to(DEV))
    step = 1e-5

    def loss(xx):
        return float((ref.norm_forward(xx, None, gamma, beta, 1e-5)[0] * dy.double()).sum())

    for i, j in ((0, 0), (1, 17), (2, 32)):
        up, down = x.double().clone(), x.double().clone()
        up[i, j] += step
        down[i, j] -= step
        diff = (loss(up) - loss(down)) / (2 * step)
        assert abs(diff - float(got["dx"][i, j])) <= 1e-4 * max(1.0, abs(diff))


# ---- gated linear recurrence ------------------------------------------------------------------


def mix_inputs(n, length, d, t, fused, starts, ragged, seed=1):
    both = torch.cat([rand((n, length, d), seed, t, 2.0, 2.0), rand((n, length, d), seed + 1, t)], 2)
    st = ln = None
    if starts:
        st = (rand((n, length), seed + 2) > 1.6).to(torch.uint8) * 3
    if ragged:
        ln = torch.tensor([[0, length, 1, length // 2, length + 7, -2][i % 6] for i in range(n)],
                          dtype=torch.int32)
        for i in range(n):
            both[i, max(0, int(ln[i])):] = float("nan")
    dev = both.to(DEV)
    g, v = dev[..., :d], dev[..., d:]
    if not fused:
        g, v = g.contiguous(), v.contiguous()
    dv = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    return g, v, both[..., :d], both[..., d:], st, ln, dv(st), dv(ln)


MIX = [
    (3, 1500, 63, True, True, True), (2, 1500, 64, False, True, False), (4, 700, 1, False, False, True),
    (1, 1, 1, False, False, False), (2, 1, 130, True, False, False), (1, 2, 3, False, True, False),
    (3, 7, 64, True, True, False), (1, 17, 33, False, False, False), (6, 40, 65, True, True, True),
    (2, 128, 128, True, False, False), (1, 129, 130, False, True, False),
    (6, 257, 31, False, True, True), (1, 1000, 5, False, False, False), (2, 2049, 12, True, True, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,length,d,fused,starts,ragged", MIX)
def test_recurrence(dtype, n, length, d, fused, starts, ragged):
    t = TYPES[dtype]
    g, v, gc, vc, st, ln, std, lnd = mix_inputs(n, length, d, t, fused, starts, ragged)
    tag = f"recurrence {dtype} {n}x{length}x{d}"
    for h0 in (rand((n, d), 9), None):
        h0d = None if h0 is None else h0.to(DEV)
        h, last = K.recurrence_forward(g, v, h0=h0d, starts=std, lens=lnd)
        want, wlast = ref.recurrence(gc, vc, h0, st, ln)
        close(h, want, CHAIN[dtype], tag + " h")
        close(last, wlast, 2e-5, tag + " last")
        dh, dl = rand((n, length, d), 10, t), rand((n, d), 11)
        if ragged:
            for i in range(n):
                dh[i, max(0, int(ln[i])):] = float("nan")
        for dlast in (dl, None):
            got = K.recurrence_backward(g, v, h, dh.to(DEV), h0=h0d,
                                        dh_last=None if dlast is None else dlast.to(DEV), starts=std,
                                        lens=lnd)
            dg, dv, dh0 = ref.recurrence_backward(gc, vc, h.cpu(), dh, h0, dlast, st, ln)
            close(got["dg"], dg, CHAIN[dtype], tag + " dg")
            close(got["dv"], dv, CHAIN[dtype], tag + " dv")
            close(got["dh0"], dh0, 2e-5, tag + " dh0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_recurrence_long_and_continued(dtype):
    """20001 tokens at once equal the same tokens in three calls that hand the state on."""
    t = TYPES[dtype]
    g, v, gc, vc, *_ = mix_inputs(1, 20001, 70, t, True, False, False)
    h, last = K.recurrence_forward(g, v)
    want, wlast = ref.recurrence(gc, vc, None, None, None)
    close(h, want, CHAIN[dtype], f"recurrence {dtype} 20001 h")
    close(last, wlast, 2e-5, f"recurrence {dtype} 20001 last")
    s, parts = None, []
    for a, b in ((0, 6000), (6000, 6001), (6001, 20001)):
        hp, s = K.recurrence_forward(g[:, a:b], v[:, a:b], h0=s)
        parts.append(hp)
    close(torch.cat(parts, 1), want, CHAIN[dtype], f"recurrence {dtype} continued h")
    close(s, wlast, 2e-5, f"recurrence {dtype} continued last")


def test_recurrence_steps_equal_the_prefill():
    g, v, gc, vc, *_ = mix_inputs(3, 9, 130, torch.bfloat16, True, False, False)
    h0 = rand((3, 130), 5).to(DEV)
    want, wlast = ref.recurrence(gc, vc, h0.cpu(), None, None)
    state = h0.clone()
    for t in range(9):
        h, out = K.recurrence_step(g[:, t], v[:, t], state, out=state)
        assert out is state
        close(h, want[:, t], 4e-3, f"recurrence step {t}")
    close(state, wlast, 2e-5, "recurrence step state")
    h, s = K.recurrence_step(g[:, 0], v[:, 0], None)
    close(h, ref.recurrence(gc[:, :1], vc[:, :1], None, None, None)[0][:, 0], 4e-3, "first step")


def test_recurrence_gate_extremes():
    """Gates at the type's lowest and largest value and at infinity: remember all or
    nothing; a document start cuts a state that is not finite."""
    length, d = 300, 8
    lo, hi = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    g = rand((1, length, d), 1)
    g[0, 50], g[0, 51], g[0, 60:90], g[0, 120] = lo, -float("inf"), float("inf"), hi
    v = rand((1, length, d), 2)
    v[0, 200, 3] = float("inf")
    st = torch.zeros((1, length), dtype=torch.uint8)
    st[0, 210] = 1
    h, last = K.recurrence_forward(g.to(DEV), v.to(DEV), starts=st.to(DEV))
    want, wlast = ref.recurrence(g, v, None, st, None)
    h, want = h.cpu().double(), want
    assert torch.equal(torch.isfinite(h), torch.isfinite(want))
    assert int((~torch.isfinite(h)).sum()) == 10   # the infinity lives until the cut
    ok = torch.isfinite(want)
    assert rel_fro(h[ok].numpy(), want[ok].numpy()) <= 2e-5
    close(last, wlast, 2e-5, "recurrence extremes last")


def test_recurrence_nan_reaches_only_its_own_channel():
    g, v, gc, vc, *_ = mix_inputs(2, 400, 20, torch.float32, False, False, False)
    v[1, 130, 7] = float("nan")
    g[0, 300, 2] = float("nan")
    h, last = K.recurrence_forward(g, v)
    want, _ = ref.recurrence(g, v, None, None, None)
    assert torch.equal(torch.isnan(h).cpu(), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert rel_fro(h.cpu().double()[ok].numpy(), want[ok].numpy()) <= 2e-5


def test_recurrence_no_tokens():
    g = torch.empty((2, 0, 5), device=DEV)
    h0, dl = rand((2, 5), 1).to(DEV), rand((2, 5), 2).to(DEV)
    h, last = K.recurrence_forward(g, g, h0=h0)
    got = K.recurrence_backward(g, g, h, g, h0=h0, dh_last=dl)
    torch.cuda.synchronize()
    assert h.shape == (2, 0, 5) and torch.equal(last, h0) and torch.equal(got["dh0"], dl)


def test_recurrence_gradient_into_a_fused_projection():
    """dg and dv written into the halves of one tensor; central differences of the forward."""
    n, length, d = 2, 150, 6
    g, v, gc, vc, *_ = mix_inputs(n, length, d, torch.float32, True, False, False)
    dh = rand((n, length, d), 4)
    h, _ = K.recurrence_forward(g, v)
    grad = torch.empty((n, length, 2 * d), device=DEV)
    K.recurrence_backward(g, v, h, dh.to(DEV), dg=grad[..., :d], dv=grad[..., d:])
    dg, dv, _ = ref.recurrence_backward(gc, vc, h.cpu(), dh, None, None, None, None)
    close(grad[..., :d], dg, 2e-5, "recurrence fused dg")
    close(grad[..., d:], dv, 2e-5, "recurrence fused dv")
    step = 1e-5
    for which, idx in (("g", (0, 3, 1)), ("g", (1, 149, 5)), ("v", (1, 0, 0)), ("v", (0, 120, 2))):
        val = []
        for sgn in (1, -1):
            gg, vv = gc.double().clone(), vc.double().clone()
            (gg if which == "g" else vv)[idx] += sgn * step
            val.append(float((ref.recurrence(gg, vv, None, None, None)[0] * dh.double()).sum()))
        diff = (val[0] - val[1]) / (2 * step)
        got = float(grad[idx[0], idx[1], idx[2] + (d if which == "v" else 0)])
        assert abs(diff - got) <= 1e-4 * max(1.0, abs(diff)), (which, idx, diff, got)


@pytest.mark.parametrize("n,length,d,starts", [(2, 3000, 300, True), (1, 60001, 43, False),
                                               (3, 5000, 64, True), (3, 5000, 65, False),
                                               (9, 5000, 517, False)])
def test_recurrence_repeats_bit_for_bit(n, length, d, starts):
    """fp32, whose last bits would show an order that depends on timing."""
    g, v, _, _, _, _, st, _ = mix_inputs(n, length, d, torch.float32, True, starts, False)
    first = K.recurrence_forward(g, v, starts=st)
    grads = K.recurrence_backward(g, v, first[0], first[0], starts=st)
    for _ in range(4):
        again = K.recurrence_forward(g, v, starts=st)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        for k, t in K.recurrence_backward(g, v, again[0], again[0], starts=st).items():
            assert torch.equal(grads[k], t), k


# ---- gated feed-forward block -------------------------------------------------------------------


def ff_tol(dtype, want):
    return 2e-2 if dtype == "bf16" and want.numel() < 64 else FF[dtype]


def ff_weights(d, f, t):
    return [w.to(t) for w in (rand((f, d), 1, std=d ** -0.5), rand((f, d), 2, std=d ** -0.5),
                              rand((d, f), 3, std=f ** -0.5))]


FF_SHAPES = [
    (1, 1, 1, 0), (1, 64, 256, 0), (2, 7, 5, 0), (3, 250, 130, 3), (16, 64, 64, 0), (17, 100, 72, 8),
    (33, 129, 257, 0), (64, 256, 640, 1), (65, 64, 128, 0), (65, 66, 130, 0), (127, 256, 640, 0),
    (130, 200, 72, 5), (257, 320, 513, 8), (300, 128, 2000, 0), (513, 1024, 576, 0),
]


# Pieces of 8 and 4 values, steps of 64 and 32 and tiles of 64 and 32 that end early in
# every operand; fewer values than a piece holds; both sides of the kernels' ranges.
FF_SHAPES += [
    (1, 8, 8, 0), (2, 9, 15, 3), (5, 31, 33, 1), (7, 63, 65, 0), (17, 8, 9, 0), (33, 71, 8, 0),
    (40, 65, 127, 3), (66, 129, 71, 0), (100, 1000, 24, 8), (64, 1023, 1025, 1), (321, 40, 4096, 0),
    (20, 5, 300, 0), (100, 300, 6, 0), (600, 901, 1100, 1), (1100, 1001, 2003, 3),
]


@pytest.mark.parametrize("dtype,n,d,f,pad", [(t, *s) for s in FF_SHAPES for t in ("bf16", "f32")]
                         + [("f32", 1100, 2000, 2001, 0)])
def test_ff(dtype, n, d, f, pad):
    t = TYPES[dtype]
    ws = ff_weights(d, f, t)
    x, dy = rand((n, d), 4, t), rand((n, d), 5, t)
    op = K.FeedForward(*[w.to(DEV) for w in ws])
    xd, dyd = wide(x, pad), wide(dy, pad)
    tag = f"ff {dtype} {n}x{d}x{f}"
    want, a, u = ref.ff_forward(x, *ws)
    close(op.forward(xd), want, ff_tol(dtype, want), tag + " y")
    y, ga, gu = op.forward(xd, save=True)
    close(y, want, ff_tol(dtype, want), tag + " y (saving)")
    close(ga, a, ff_tol(dtype, a), tag + " a")
    close(gu, u, ff_tol(dtype, u), tag + " u")
    got = op.backward(xd, ga, gu, dyd)
    for name, w in zip(("dx", "dw_gate", "dw_up", "dw_down"), ref.ff_backward(x, *ws, dy)):
        close(got[name], w, ff_tol(dtype, w), f"{tag} {name}")


@pytest.mark.parametrize("n", [1, 8, 64, 200, 1000])
def test_ff_layer_shape(n):
    """The 4B-shaped block; reference products in fp32 on the GPU's host."""
    d, f = 2560, 9728
    ws = ff_weights(d, f, torch.bfloat16)
    x = rand((n, d), 4, torch.bfloat16)
    op = K.FeedForward(*[w.to(DEV) for w in ws])
    y = op.forward(x.to(DEV))
    xs, (wg, wu, wd) = x.float(), [w.float() for w in ws]
    a, u = xs @ wg.T, xs @ wu.T
    close(y, ((a * torch.sigmoid(a) * u) @ wd.T).double(), 8e-3, f"ff 4B-shaped n={n}")


def test_ff_large_backward():
    """Enough tokens for the large tiles in every product."""
    n, d, f = 2048, 2048, 4096
    ws = [w.to(DEV) for w in ff_weights(d, f, torch.bfloat16)]
    x, dy = rand((n, d), 4, torch.bfloat16).to(DEV), rand((n, d), 5, torch.bfloat16).to(DEV)
    op = K.FeedForward(*ws)
    y, a, u = op.forward(x, save=True)
    got = op.backward(x, a, u, dy)
    xf, wg, wu, wd, dyf = x.float(), *[w.float() for w in ws], dy.float()
    af, uf = xf @ wg.T, xf @ wu.T
    s = torch.sigmoid(af)
    z, dz = af * s * uf, dyf @ wd
    da, du = dz * uf * (s + af * s * (1 - s)), dz * af * s
    close(y, (z @ wd.T).double().cpu(), 8e-3, "ff large y")
    for name, w in (("dx", da @ wg + du @ wu), ("dw_gate", da.T @ xf), ("dw_up", du.T @ xf),
                    ("dw_down", dyf.T @ z)):
        close(got[name], w.double().cpu(), 8e-3, f"ff large {name}")


def test_ff_no_tokens():
    for t in (torch.bfloat16, torch.float32):
        op = K.FeedForward(*[w.to(DEV) for w in ff_weights(5, 7, t)])
        e = torch.empty((0, 5), dtype=t, device=DEV)
        y, a, u = op.forward(e, save=True)
        got = op.backward(e, a, u, e)
        torch.cuda.synchronize()
        assert y.shape == (0, 5)
        assert all(float(got[k].float().abs().max()) == 0.0 for k in ("dw_gate", "dw_up", "dw_down"))


def test_ff_keeps_rows_apart():
    """A token that is not finite reaches its own row alone (both size regimes)."""
    ws = [w.to(DEV) for w in ff_weights(128, 256, torch.bfloat16)]
    op = K.FeedForward(*ws)
    for n in (20, 150):
        x = rand((n, 128), 4, torch.bfloat16).to(DEV)
        base = op.forward(x)
        x[7, 3] = float("nan")
        y = op.forward(x)
        keep = [i for i in range(n) if i != 7]
        assert torch.equal(y[keep], base[keep]) and torch.isnan(y[7]).all()


def test_ff_gradient_against_differences():
    n, d, f = 4, 12, 20
    ws = ff_weights(d, f, torch.float32)
    x, dy = rand((n, d), 4), rand((n, d), 5)
    op = K.FeedForward(*[w.to(DEV) for w in ws])
    _, a, u = op.forward(x.to(DEV), save=True)
    got = op.backward(x.to(DEV), a, u, dy.to(DEV))
    step = 1e-5
    args = [x.double()] + [w.double() for w in ws]
    for k, (name, idx) in enumerate((("dx", (1, 3)), ("dw_gate", (5, 2)), ("dw_up", (19, 11)),
                                     ("dw_down", (0, 7)))):
        val = []
        for sgn in (1, -1):
            moved = [t.clone() for t in args]
            moved[k][idx] += sgn * step
            val.append(float((ref.ff_forward(*moved)[0] * dy.double()).sum()))
        diff = (val[0] - val[1]) / (2 * step)
        assert abs(diff - float(got[name][idx])) <= 1e-4 * max(1.0, abs(diff)), name


# ---- large offsets, repeatability ---------------------------------------------------------------------


def test_more_blocks_than_an_axis_takes():
    """Narrow rows in numbers that, a few threads each, pass 2^32 threads in a line."""
    n = (1 << 26) + 9
    x = torch.empty((n, 3), dtype=torch.bfloat16, device=DEV).normal_()
    op = K.Norm(torch.ones(3, dtype=torch.bfloat16, device=DEV), None)
    y, _, mean, rstd = op.forward(x)
    for at in (0, (1 << 22) - 7, (1 << 25) + 1, n - 5000):
        part = slice(at, at + 5000)
        yp, _, mp, rp = op.forward(x[part])
        assert torch.equal(y[part], yp) and torch.equal(mean[part], mp) and torch.equal(rstd[part], rp)
    del x, y, mean, rstd

    batch, length = 65535, 128 * 128 + 3   # 129 tiles a sequence
    g = torch.empty((batch, length, 1), dtype=torch.bfloat16, device=DEV).normal_().add_(3.0)
    v = torch.empty_like(g).normal_()
    h, last = K.recurrence_forward(g, v)
    got = K.recurrence_backward(g, v, h, h)
    for i in (0, 1, 31000, batch - 1):
        one = slice(i, i + 1)
        hp, lp = K.recurrence_forward(g[one], v[one])
        assert torch.equal(h[one], hp) and torch.equal(last[one], lp)
        for k, t in K.recurrence_backward(g[one], v[one], hp, hp).items():
            assert torch.equal(got[k][one], t), (i, k)
    del g, v, h, last, got

    n = (1 << 20) + 77
    W = [rand(s, i, torch.bfloat16, s[1] ** -0.5).to(DEV) for i, s in enumerate(((16, 8), (16, 8), (8, 16)))]
    ff, x = K.FeedForward(*W), torch.empty((n, 8), dtype=torch.bfloat16, device=DEV).normal_()
    y = ff.forward(x)
    y20 = ff.forward(x[:1 << 20])
    for at in (0, 500000, (1 << 20) - 3000, n - 3000):
        part = slice(at, at + 3000)
        want = ff.forward(x[part]).float().cpu().numpy()
        # the same roundings (z, y to bf16) of sums in another order
        assert rel_fro(y[part].float().cpu().numpy(), want) <= 4e-3, at
        if part.stop <= 1 << 20:
            assert rel_fro(y20[part].float().cpu().numpy(), want) <= 4e-3, at


def test_norm_offsets_past_32_bits():
    """1.1 M rows of 2048: the last rows' results equal those of the rows alone."""
    n, d = 1100000, 2048
    assert n * d > 1 << 31
    x = torch.empty((n, d), dtype=torch.bfloat16, device=DEV).normal_()
    op = K.Norm(torch.ones(d, dtype=torch.bfloat16, device=DEV), torch.zeros(d, dtype=torch.bfloat16, device=DEV))
    y, h, mean, rstd = op.forward(x, x)
    tail = slice(n - 5000, n)
    yt, ht, mt, rt = op.forward(x[tail], x[tail])
    assert torch.equal(y[tail], yt) and torch.equal(h[tail], ht) and torch.equal(mean[tail], mt)
    dx = op.backward(h, mean, rstd, y, x)["dx"]
    want = op.backward(ht, mt, rt, yt, x[tail])["dx"]   # fewer rows: another split of a row's sum
    assert rel_fro(dx[tail].float().cpu().numpy(), want.float().cpu().numpy()) <= 4e-3


def test_recurrence_offsets_past_32_bits():
    """1.1 M tokens of 2048 channels in one sequence; the last tokens equal a run from
    the state before them (gates near 1/4: what is 100 tokens old has gone)."""
    length, d = 1100000, 2048
    assert length * d > 1 << 31
    both = torch.empty((1, length, 2 * d), dtype=torch.bfloat16, device=DEV)
    for at in range(0, length, 100000):   # in pieces: torch's own indexing has its limits
        both[:, at:at + 100000].normal_()
    g, v = both[..., :d], both[..., d:]
    for at in range(0, length, 100000):
        g[:, at:at + 100000] -= 1
    h, last = K.recurrence_forward(g, v)
    cut = length - 3000
    ht, lt = K.recurrence_forward(g[:, cut:], v[:, cut:])
    assert rel_fro(h[:, -2000:].float().cpu().numpy(), ht[:, -2000:].float().cpu().numpy()) <= 4e-3
    assert rel_fro(last.cpu().numpy(), lt.cpu().numpy()) <= 2e-5
    got = K.recurrence_backward(g, v, h, h)
    want = K.recurrence_backward(g[:, cut:], v[:, cut:], h[:, cut:], h[:, cut:],
                                 h0=h[:, cut - 1].float().contiguous())
    for k in ("dg", "dv"):
        assert rel_fro(got[k][:, cut:].float().cpu().numpy(), want[k].float().cpu().numpy()) <= 4e-3


def test_ff_offsets_past_32_bits():
    """262144 tokens through d_ff 9728: z, a, u and their gradients pass 2^31 elements."""
    n, d, f = 262144, 64, 9728
    assert n * f > 1 << 31
    op = K.FeedForward(*[w.to(DEV) for w in ff_weights(d, f, torch.bfloat16)])
    x = torch.empty((n, d), dtype=torch.bfloat16, device=DEV).normal_()
    dy = torch.empty((n, d), dtype=torch.bfloat16, device=DEV).normal_()
    y, a, u = op.forward(x, save=True)
    dx = op.backward(x, a, u, dy)["dx"]
    tail = slice(n - 300, n)
    yt, at, ut = op.forward(x[tail], save=True)
    assert rel_fro(y[tail].float().cpu().numpy(), yt.float().cpu().numpy()) <= 8e-3
    assert rel_fro(a[tail].cpu().numpy(), at.cpu().numpy()) <= 1e-5
    dxt = op.backward(x[tail], at, ut, dy[tail])["dx"]
    assert rel_fro(dx[tail].float().cpu().numpy(), dxt.float().cpu().numpy()) <= 8e-3


def test_norm_and_ff_repeat_bit_for_bit():
    x, dy = rand((3000, 512), 1, torch.bfloat16).to(DEV), rand((3000, 512), 2, torch.bfloat16).to(DEV)
    norm = K.Norm(torch.ones(512, dtype=torch.bfloat16, device=DEV))
    ff = K.FeedForward(*[w.to(DEV) for w in ff_weights(512, 640, torch.bfloat16)])

    def run():
        y, h, m, r = norm.forward(x, dy)
        z, a, u = ff.forward(y, save=True)
        return [y, z, *norm.backward(h, m, r, dy).values(), *ff.backward(y, a, u, dy).values()]

    first = run()
    for _ in range(2):
        for p, q in zip(first, run()):
            assert torch.equal(p, q)


# ---- streams and graphs ---------------------------------------------------------------------------


def test_calls_on_another_stream():
    """Inputs produced and consumed on a side stream; temporaries are not reused under it."""
    s = torch.cuda.Stream()
    ws = [w.to(DEV) for w in ff_weights(192, 320, torch.bfloat16)]
    op = K.FeedForward(*ws)
    x = rand((300, 192), 4, torch.bfloat16).to(DEV)
    g = rand((1, 4000, 192), 6, torch.bfloat16, 2.0, 2.0).to(DEV)
    want, wanth = op.forward(x), K.recurrence_forward(g, g)[0]
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        y = op.forward(x, stream=s)
        h, _ = K.recurrence_forward(g, g, stream=s)
        junk = torch.full((1 << 20,), 7.0, device=DEV)   # would land in freed workspace
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want) and torch.equal(h, wanth)
        del junk


def test_block_in_a_graph():
    """norm, recurrence and feed-forward captured once and replayed on new inputs."""
    d, f, n, length = 128, 320, 2, 700
    ws = [w.to(DEV) for w in ff_weights(d, f, torch.bfloat16)]
    op = K.FeedForward(*ws)
    norm = K.Norm(torch.ones(d, dtype=torch.bfloat16, device=DEV))
    x = torch.empty((n, length, d), dtype=torch.bfloat16, device=DEV)

    def block():
        y, _, _, _ = norm.forward(x)
        h, last = K.recurrence_forward(y, y)
        z, hh, _, _ = norm.forward(x, h)
        return op.forward(z), last

    x.copy_(rand(x.shape, 1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, last = block()
    for seed in (2, 3, 4, 5):
        x.copy_(rand(x.shape, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = (out.clone(), last.clone())
        want = block()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), seed

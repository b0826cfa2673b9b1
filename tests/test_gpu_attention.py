"""The attention operators against 64 bits (attention_reference.py): types, head layouts,
lengths, strides, masks, pages, what is not finite, and the operators together."""
from __future__ import annotations

import math

import pytest
import torch

import attention_reference as R
from chunked_weight_mlp_amd import attention as A
from parity_check import report

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.load()


def rand(shape, seed, dtype=F32, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)


WORST = {}


@pytest.fixture(scope="module", autouse=True)
def worst_shares():
    yield
    for name in sorted(WORST):
        report(f"[attention] {name}: {WORST[name]:.3f} of the bound at worst")


def within(name, got, want, bound):
    """Every element within its bound; the worst share of it is reported at the end."""
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    worst = (err / bound.clamp_min(1e-30)).max().item() if err.numel() else 0.0
    key = name.split(" (")[0] + f" {got.dtype}"[:12]
    WORST[key] = max(WORST.get(key, 0.0), worst)
    assert worst <= 1.0, (name, worst, err.max().item())


def offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)


def layout(t, kind, seed):
    """The same values, laid out otherwise: a slice of a wider tensor, heads outermost, rows
    that start anywhere."""
    n, h, d = t.shape
    if kind == "dense":
        return t
    if kind == "slice":
        wide = rand((n, h * d + 8 * d), seed, t.dtype)
        wide[:, 4 * d:4 * d + h * d] = t.reshape(n, -1)
        return wide[:, 4 * d:4 * d + h * d].view(n, h, d)
    if kind == "heads":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    wide = rand((n, h, d + 3), seed, t.dtype)   # odd
    wide[..., 1:d + 1] = t
    return wide[..., 1:d + 1]


LAYOUTS = ("dense", "slice", "heads", "odd")

# ---- head norm --------------------------------------------------------------------------

HEADS = [  # hq, hk, dh, rotary, interleaved, gammas
    (4, 2, 128, 128, False, "qk"), (4, 4, 64, 64, True, "qk"), (3, 1, 72, 24, True, "qk"),
    (5, 1, 80, 80, False, "q"), (2, 2, 33, 32, False, "qk"), (1, 1, 1, 0, False, "k"), (7, 7, 40, 20, False, ""),
    (2, 1, 128, 64, True, "qk"), (9, 3, 127, 126, False, "qk"), (2, 1, 2, 2, False, "qk"), (1, 1, 96, 48, False, "qk"),
]


def head_op(hq, hk, dh, rotary, interleaved, gammas, dtype, theta=1e4):
    inv = theta ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1)).to(DEV)
    gq, gk = (rand((dh,), s, dtype, 0.3, 1.0) if c in gammas else None for s, c in ((1, "q"), (2, "k")))
    return A.HeadNorm(gq, gk, inv, eps=EPS, interleaved=interleaved, head_dim=dh, dtype=dtype), gq, gk, inv


def head_bound(x, gamma, want, dtype, angle=4 * R.E32):
    """One rounding to the type; in fp32 the norm's few roundings of each channel, and of the
    pair's other one through the rotation (angles within `angle`)."""
    n = R.w64(x)
    if gamma is not None:
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS) * R.w64(gamma)
    size = n.abs().amax(-1, keepdim=True)
    return R.half_step(dtype) * want.abs() * 1.01 + (angle + 16 * R.E32 + x.shape[-1] * R.E32) * 2 * size + 1e-37


@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", HEADS)
def test_heads_forward(case, dtype, kind):
    hq, hk, dh = case[:3]
    op, gq, gk, inv = head_op(*case, dtype)
    for n in (1, 3, 130):
        q, k = layout(rand((n, hq, dh), 3, dtype), kind, 5), layout(rand((n, hk, dh), 4, dtype, 3.0), kind, 6)
        pos = torch.randint(-5, 131072, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).to(DEV)
        got = op.forward(q, k, pos)
        for name, x, g, y in (("q", q, gq, got[0]), ("k", k, gk, got[1])):
            want = R.head_forward(x, g, pos, inv, EPS, case[4])
            within(f"heads forward {name} {case} {n}", y, want, head_bound(x, g, want, dtype))
            assert y.is_contiguous()


def test_heads_far_positions():
    """Angles of positions near 2^31 are those of 64 bits."""
    op, gq, gk, inv = head_op(2, 1, 64, 64, False, "qk", F32)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0], dtype=torch.int32, device=DEV)
    q, k = rand((4, 2, 64), 1), rand((4, 1, 64), 2)
    got = op.forward(q, k, pos)
    for x, g, y in ((q, gq, got[0]), (k, gk, got[1])):
        want = R.head_forward(x, g, pos, inv, EPS, False)
        # pos inv_freq in 64 bits: half a step of 2^31, 2.4e-7, on either side
        within("heads far", y, want, head_bound(x, g, want, F32, angle=4 * R.E32 + 5e-7))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", HEADS)
def test_heads_backward(case, dtype):
    hq, hk, dh = case[:3]
    op, gq, gk, inv = head_op(*case, dtype)
    for n, kind in ((1, "dense"), (3, "odd"), (517, "slice"), (130, "heads")):
        q, k = layout(rand((n, hq, dh), 3, dtype), kind, 5), layout(rand((n, hk, dh), 4, dtype, 3.0), kind, 6)
        dq, dk = layout(rand((n, hq, dh), 7, dtype), kind, 9), layout(rand((n, hk, dh), 8, dtype), kind, 10)
        pos = torch.arange(n, dtype=torch.int32, device=DEV) + 4000
        got = op.backward(q, k, pos, dq, dk)
        for name, x, g, dy in (("q", q, gq, dq), ("k", k, gk, dk)):
            dx, dg = R.head_backward(x, g, pos, inv, EPS, case[4], dy)
            r = 1 / torch.sqrt((R.w64(x) ** 2).mean(-1, keepdim=True) + EPS) if g is not None else 1.0
            size = (R.w64(dy).abs().amax(-1, keepdim=True) * (1 if g is None else g.double().abs().max()) * r)
            big = (R.w64(x).abs() * r).amax(-1, keepdim=True) if g is not None else 1.0
            bound = (R.half_step(dtype) * dx.abs() * 1.01 + (32 + 2 * dh) * R.E32 * 2 * size * (1 + big * big) + 1e-37)
            within(f"heads backward d{name} {case} {n}", got["d" + name], dx, bound)
            if g is None:
                assert got[f"d{name}_gamma"] is None
                continue
            terms = (R.rotate(R.w64(dy), pos, inv, case[4], True).abs() * R.w64(x).abs() * r).sum((0, 1))
            worst = (R.w64(dy).abs().amax() * R.w64(x).abs() * r).sum((0, 1))
            within(f"heads backward d{name}_gamma {case} {n}", got[f"d{name}_gamma"], dg,
                   R.E32 * (48 * terms + 8 * worst) + 1e-30)


def test_heads_backward_against_differences():
    """The fp32 gradients against central differences of the formula in 64 bits."""
    case = (2, 1, 24, 16, False, "qk")
    op, gq, gk, inv = head_op(*case, F32)
    q, k, dq, dk = rand((3, 2, 24), 1), rand((3, 1, 24), 2), rand((3, 2, 24), 3), rand((3, 1, 24), 4)
    pos = torch.tensor([0, 7, 1000], dtype=torch.int32, device=DEV)
    got = op.backward(q, k, pos, dq, dk)

    def loss(x, g, dy):
        return (R.head_forward(x, g, pos, inv, EPS, False) * dy.double()).sum()

    for x, g, dy, dx, dg in ((q, gq, dq, got["dq"], got["dq_gamma"]), (k, gk, dk, got["dk"], got["dk_gamma"])):
        x, g, step = x.double(), g.double(), 1e-5
        for t, d in ((x, dx), (g, dg)):
            for i in range(0, t.numel(), 5):
                at = t.view(-1)[i].item()
                t.view(-1)[i] = at + step
                up = loss(x, g, dy)
                t.view(-1)[i] = at - step
                down = loss(x, g, dy)
                t.view(-1)[i] = at
                # the difference's own error: step^2 times third derivatives of order 10
                assert abs((up - down).item() / (2 * step) - d.view(-1)[i].item()) <= 2e-5


def test_heads_no_tokens():
    op, *_ = head_op(2, 1, 64, 64, False, "qk", BF16)
    q, k = rand((0, 2, 64), 1, BF16), rand((0, 1, 64), 2, BF16)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    assert op.forward(q, k, pos)[0].shape == (0, 2, 64)
    got = op.backward(q, k, pos, q, k)
    assert (got["dq_gamma"] == 0).all() and (got["dk_gamma"] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hk,dh,page", [(4, 2, 128, 16), (3, 3, 72, 5), (8, 1, 33, 1), (2, 2, 64, 64)])
def test_append(hq, hk, dh, page, dtype):
    """q and k as the forward's; v bit for bit; everything else in the cache as it was."""
    op, *_ = head_op(hq, hk, dh, dh // 2 * 2, False, "qk", dtype)
    batch, width, n = 3, 4, 9
    pages = batch * width
    cache = A.KVCache(rand((pages, hk, page, dh), 1, dtype), rand((pages, hk, page, dh), 2, dtype))
    before = cache.k.clone(), cache.v.clone()
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(batch, width)
    table[1, 0], table[2, 0] = -1, pages
    wide = torch.full((batch, width + 2), 99, dtype=torch.int32)
    wide[:, :width] = table
    seqs = torch.tensor([0, 0, 1, 1, 2, 5, -1, 2, 0], dtype=torch.int32)
    pos = torch.tensor([0, page, 0, 2 * page, 0, 1, 1, -1, width * page], dtype=torch.int32)
    qkv = rand((n, (hq + 2 * hk) * dh), 4, dtype)
    q, k, v = (t.view(n, -1, dh) for t in qkv.split([hq * dh, hk * dh, hk * dh], 1))
    got = op.append(q, k, v, pos.to(DEV), cache, wide.to(DEV)[:, :width], seqs.to(DEV))
    qq, kk = op.forward(q, k, pos.to(DEV))
    assert torch.equal(got, qq)
    want_k, want_v = before
    written = 0
    for t in range(n):
        s, p = int(seqs[t]), int(pos[t])
        if not (0 <= s < batch and 0 <= p < width * page):
            continue
        at = int(table[s, p // page])
        if 0 <= at < pages:
            want_k[at, :, p % page], want_v[at, :, p % page] = kk[t], v[t]
            written += 1
    assert written == 3 and torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
    # without seqs: token t is sequence t's
    first = torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV)
    good = table.clone()
    good[1, 0], good[2, 0] = 2, 3
    good[0, 0] = 1
    op.append(q[:3], k[:3], v[:3], first, cache, good.to(DEV))
    at = torch.tensor([good[i, 1 // page] for i in range(3)], device=DEV).long()
    _, kk = op.forward(q[:3], k[:3], first)
    assert torch.equal(cache.k[at, :, 1 % page], kk) and torch.equal(cache.v[at, :, 1 % page], v[:3])


# ---- attention over prompts -------------------------------------------------------------

PROMPTS = [  # lens of queries, of keys, hq, hk, dh, causal, window
    ([1], [1], 1, 1, 64, True, 0),
    ([300], [300], 4, 2, 128, True, 0),
    ([7, 0, 65, 256, 31], None, 4, 4, 64, True, 0),
    ([129, 513], None, 6, 2, 40, True, 0),
    ([64, 20], [300, 64], 2, 1, 72, True, 0),        # keys from before
    ([100, 5], [40, 0], 2, 2, 128, True, 0),         # queries that see no key
    ([200, 3], [77, 130], 3, 1, 33, False, 0),       # every key
    ([400, 90], None, 2, 1, 128, True, 1),           # itself alone
    ([600], [700], 2, 2, 96, True, 100),
    ([257], None, 8, 1, 128, True, 64),
    ([5] * 70, None, 2, 1, 64, True, 0),             # more sequences than lanes
    ([1000], None, 5, 5, 80, True, 0),
    ([2, 1], [2, 1], 2, 1, 1, True, 0),
    ([33], [1500], 4, 1, 128, True, 700),
]


def prompt(case, dtype, kind="dense", tail=0, std=2.0):
    lq, lk, hq, hk, dh, causal, window = case
    lk = lq if lk is None else lk
    n, nk = sum(lq) + tail, sum(lk) + tail
    q = layout(rand((n, hq, dh), 1, dtype, std), kind, 11)
    k, v = layout(rand((nk, hk, dh), 2, dtype), kind, 12), layout(rand((nk, hk, dh), 3, dtype), kind, 13)
    dy = layout(rand((n, hq, dh), 4, dtype), kind, 14)
    how = dict(offsets=offsets(lq), k_offsets=offsets(lk), causal=causal, window=window)
    return q, k, v, dy, lq, lk, how


@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", PROMPTS)
def test_prompt(case, dtype, kind):
    """Forward and backward; rows behind the last sequence are zero."""
    tail = 0 if kind == "dense" else 37
    q, k, v, dy, lq, lk, how = prompt(case, dtype, kind, tail)
    o, lse = A.attention_forward(q, k, v, **how)
    want, want_lse, bound, lse_bound = R.attention(q, k, v, lq, lk, how["causal"], how["window"])
    within(f"prompt o {case[:5]}", o, want, bound)
    none = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all()
    within(f"prompt lse {case[:5]}", lse[~none], want_lse[~none], lse_bound[~none])
    got = A.attention_backward(q, k, v, o, lse, dy, **how)
    want, bound = R.attention_backward(q, k, v, o, lse, dy, lq, lk, how["causal"], how["window"])
    for x in want:
        within(f"prompt {x} {case[:5]}", got[x], want[x], bound[x])
        m = sum(lq if x == "dq" else lk)
        assert (got[x][m:] == 0).all() and got[x].is_contiguous()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_one_sequence_without_offsets(dtype):
    q, k, v, dy, lq, lk, how = prompt(([150], [200], 4, 2, 64, True, 0), dtype)
    o, lse = A.attention_forward(q, k, v, **how)
    assert torch.equal(A.attention_forward(q, k, v)[0], o)
    got, want = A.attention_backward(q, k, v, o, lse, dy), A.attention_backward(q, k, v, o, lse, dy, **how)
    assert all(torch.equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_prompt_scale(scale, dtype):
    q, k, v, dy, lq, lk, how = prompt(([150], [200], 4, 2, 64, True, 0), dtype, std=1.0)
    o, lse = A.attention_forward(q, k, v, scale=scale, **how)
    want, want_lse, bound, lse_bound = R.attention(q, k, v, lq, lk, scale=scale)
    within("prompt scale o", o, want, bound)
    within("prompt scale lse", lse, want_lse, lse_bound)
    got = A.attention_backward(q, k, v, o, lse, dy, scale=scale, **how)
    want, bound = R.attention_backward(q, k, v, o, lse, dy, lq, lk, scale=scale)
    for x in want:
        within(f"prompt scale {x}", got[x], want[x], bound[x] + 1e-30)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 50])
def test_prompt_what_is_not_seen_does_not_count(window, dtype, value):
    """Rows of q, k, v and dy that are not finite: every result that does not see them is bit
    for bit what it is with other values there, and what sees them is not finite."""
    case = ([300, 90, 60], None, 4, 2, 128, True, window)
    q, k, v, dy, lq, lk, how = prompt(case, dtype, tail=5)
    o, lse = A.attention_forward(q, k, v, **how)
    grads = A.attention_backward(q, k, v, o, lse, dy, **how)
    at = 170
    sees = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)     # queries that see key 170
    sees[at:at + window if window else 300] = True
    for t in "kv":
        bad = dict(k=k.clone(), v=v.clone())
        bad[t][at, 1, 5 if t == "v" else slice(None)] = value
        bad[t][-5:] = value
        oo, ll = A.attention_forward(q, bad["k"], bad["v"], **how)
        assert torch.equal(oo[~sees], o[~sees]) and torch.equal(ll[:, ~sees], lse[:, ~sees])
        assert torch.equal(oo[:, :2], o[:, :2])                       # the other key head's
        if t == "v":
            assert not torch.isfinite(oo[sees][:, 2:, 5]).any()
            assert torch.equal(torch.cat([oo[:, 2:, :5], oo[:, 2:, 6:]], -1), torch.cat([o[:, 2:, :5], o[:, 2:, 6:]], -1))
        elif value != value:
            assert not torch.isfinite(oo[sees][:, 2:]).any()
        got = A.attention_backward(q, bad["k"], bad["v"], oo, ll, dy, **how)
        assert torch.equal(got["dq"][~sees], grads["dq"][~sees])
        if t == "v" or value != value:
            assert not torch.isfinite(got["dq"][sees][:, 2:]).all(-1).any()
    seen_by = torch.zeros(k.shape[0], dtype=torch.bool, device=DEV)  # keys that query 170 sees
    seen_by[max(0, at - window + 1) if window else 0:at + 1] = True
    for t in ("q", "dy"):
        bad = dict(q=q.clone(), dy=dy.clone())
        bad[t][at, 2] = value
        bad[t][-5:] = value
        oo, ll = A.attention_forward(bad["q"], k, v, **how)
        keep = torch.arange(q.shape[0], device=DEV) != at
        keep[-5:] = False
        assert torch.equal(oo[keep], o[keep]) and torch.equal(oo[-5:], torch.zeros_like(oo[-5:]))
        got = A.attention_backward(bad["q"], k, v, oo, ll, bad["dy"], **how)
        assert torch.equal(got["dq"][keep], grads["dq"][keep])
        for x in ("dk", "dv"):
            assert torch.equal(got[x][~seen_by], grads[x][~seen_by]), (t, x)
            assert torch.equal(got[x][:, 0], grads[x][:, 0])
            assert not torch.isfinite(got[x][seen_by][:, 1]).all(-1).any(), (t, x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hk,dh", [(4, 2, 128), (2, 1, 64), (3, 3, 72), (2, 2, 33)])
def test_prompt_one_key(hq, hk, dh, dtype):
    """A query that sees one key: o is its v and the gradients through the softmax are zero, to
    the bit, in sequences of one token, behind a window of one and in the first row."""
    q, k, v, dy, lq, lk, how = prompt(([1] * 5 + [70], None, hq, hk, dh, True, 1), dtype)
    o, lse = A.attention_forward(q, k, v, **how)
    assert torch.equal(o, v.repeat_interleave(hq // hk, 1))
    got = A.attention_backward(q, k, v, o, lse, dy, **how)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    how["window"] = 0
    o, lse = A.attention_forward(q, k, v, **how)
    got = A.attention_backward(q, k, v, o, lse, dy, **how)
    assert (got["dq"][:6] == 0).all() and (got["dk"][:5] == 0).all()
    assert torch.equal(o[:6], v[:6].repeat_interleave(hq // hk, 1))


def test_prompt_large_scores():
    """Scores far from zero, rising along the keys: the running maximum moves all the time."""
    n, dh = 700, 64
    for dtype in (BF16, F32):
        q = torch.ones((n, 1, dh), device=DEV, dtype=dtype)
        k = (torch.arange(n, device=DEV, dtype=torch.float32)[:, None, None] / 16 - 20).expand(n, 1, dh).to(dtype).contiguous()
        v = rand((n, 1, dh), 1, dtype)
        for kk in (k, -k):
            o, lse = A.attention_forward(q, kk, v)
            want, want_lse, bound, lse_bound = R.attention(q, kk, v, [n], [n])
            within("large scores o", o, want, bound)
            within("large scores lse", lse, want_lse, lse_bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_longer(dtype):
    """Several thousand tokens in sequences that end anywhere, grouped heads."""
    q, k, v, dy, lq, lk, how = prompt(([2500, 1, 1300, 700], None, 4, 2, 128, True, 0), dtype)
    o, lse = A.attention_forward(q, k, v, **how)
    want, want_lse, bound, lse_bound = R.attention(q, k, v, lq, lk)
    within("longer o", o, want, bound)
    got = A.attention_backward(q, k, v, o, lse, dy, **how)
    want, bound = R.attention_backward(q, k, v, o, lse, dy, lq, lk)
    for x in want:
        within(f"longer {x}", got[x], want[x], bound[x])
        # and together much nearer than each rounding's worst case
        rel = ((got[x].double() - want[x]).norm() / want[x].norm()).item()
        report(f"[attention] longer {x} {dtype}: rel {rel:.2e}")
        assert rel <= (4e-3 if dtype is BF16 else 2e-6)


def test_prompt_gradients_against_differences():
    lq, lk = [9, 4], [12, 4]
    q, k, v, dy = rand((13, 2, 8), 1), rand((16, 1, 8), 2), rand((16, 1, 8), 3), rand((13, 2, 8), 4)
    how = dict(offsets=offsets(lq), k_offsets=offsets(lk), window=6)
    o, lse = A.attention_forward(q, k, v, **how)
    got = A.attention_backward(q, k, v, o, lse, dy, **how)
    t64 = [t.double() for t in (q, k, v)]

    def loss():
        return (R.attention(*t64, lq, lk, True, 6)[0] * dy.double()).sum().item()

    step = 1e-5
    for t, d in zip(t64, (got["dq"], got["dk"], got["dv"])):
        for i in range(0, t.numel(), 7):
            at = t.view(-1)[i].item()
            t.view(-1)[i] = at + step
            up = loss()
            t.view(-1)[i] = at - step
            down = loss()
            t.view(-1)[i] = at
            assert abs((up - down) / (2 * step) - d.view(-1)[i].item()) <= 2e-5


def test_prompt_offsets_that_are_no_offsets():
    """Offsets outside the tensors are cut to them, falling ones give empty sequences."""
    q, k, v = rand((50, 2, 64), 1, BF16), rand((50, 1, 64), 2, BF16), rand((50, 1, 64), 3, BF16)
    off = torch.tensor([7, 30, 10 ** 9], dtype=torch.int32, device=DEV)
    o, _ = A.attention_forward(q, k, v, offsets=off)
    want, _ = A.attention_forward(q, k, v, offsets=torch.tensor([0, 30, 50], dtype=torch.int32, device=DEV))
    assert torch.equal(o, want)
    n = 2000
    q, k, v = rand((n, 2, 64), 1, BF16), rand((n, 1, 64), 2, BF16), rand((n, 1, 64), 3, BF16)
    for off in ([0, 40, 20, -5], [0, 1000, 0, 1000], [0, 2000, 1000, 3000, 0, 1], [5, 4, 3, 2, 1, 0]):
        off = torch.tensor(off, dtype=torch.int32, device=DEV)
        o, lse = A.attention_forward(q, k, v, offsets=off)
        A.attention_backward(q, k, v, o, lse, q, offsets=off)
        torch.cuda.synchronize()


def test_prompt_no_sequence():
    """Offsets of no sequence: every row is behind the last one."""
    q, k = rand((300, 2, 64), 1, BF16), rand((300, 1, 64), 2, BF16)
    off = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = A.attention_forward(q, k, k, offsets=off)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert all((t == 0).all() for t in A.attention_backward(q, k, k, o, lse, q, offsets=off).values())


def test_prompt_empty():
    for lq, lk in (([0], [0]), ([0, 0], [3, 4]), ([3, 4], [0, 0])):
        q, k = rand((sum(lq), 2, 64), 1, BF16), rand((sum(lk), 1, 64), 2, BF16)
        how = dict(offsets=offsets(lq), k_offsets=offsets(lk))
        o, lse = A.attention_forward(q, k, k, **how)
        assert (o == 0).all() and (lse == -math.inf).all()
        got = A.attention_backward(q, k, k, o, lse, q, **how)
        assert all((t == 0).all() for t in got.values())


# ---- one new token over the paged cache ---------------------------------------------------


def paged(lens, hk, dh, page, dtype, seed=1, width=None, spare=2):
    """A cache whose slots behind the sequences hold NaN, and its table."""
    need = [-(-m // page) for m in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max([1, width or 1] + need)), -1, dtype=torch.int32)
    at = 0
    k, v = (torch.full((pages, hk, page, dh), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    for i, m in enumerate(lens):
        mine = order[at:at + need[i]]
        table[i, :need[i]] = mine
        at += need[i]
        if m:
            for t, s in ((k, 10), (v, 20)):
                x = rand((m, hk, dh), s + i, dtype)
                slot = torch.arange(m)
                t[mine[slot // page].long().to(DEV), :, (slot % page).to(DEV)] = x
    return A.KVCache(k, v), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


STEPS = [  # lens, hq, hk, dh, page, window
    ([1], 1, 1, 64, 16, 0),
    ([1, 0, 17, 128, 129], 4, 2, 128, 16, 0),
    ([5, 300, 77], 6, 3, 72, 24, 0),
    ([1000, 3, 4096, 0, 511], 8, 2, 128, 64, 0),
    ([640, 2000], 2, 2, 33, 1, 0),
    ([900, 40], 5, 1, 80, 128, 100),
    ([2049], 40, 1, 128, 64, 0),                  # a group of more heads than a tile has columns
    ([700, 701, 0, 0, 1], 66, 2, 40, 7, 33),
    ([9000], 4, 4, 96, 256, 0),
    ([0, 0], 2, 1, 64, 16, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide", [0, 300])
@pytest.mark.parametrize("case", STEPS)
def test_step(case, wide, dtype):
    lens, hq, hk, dh, page, window = case
    cache, table, n = paged(lens, hk, dh, page, dtype, width=wide or None)
    q = rand((len(lens), hq, dh), 5, dtype, 2.0)
    for kind in LAYOUTS:
        o = A.attention_step(layout(q, kind, 6), cache, table, n, window=window)
        want, bound = R.step(q, cache.k, cache.v, table, n, window)
        within(f"step {case}", o, want, bound)


def test_step_many_sequences():
    """More sequences than lanes, most of them short."""
    lens = [(i * 37) % 100 for i in range(150)] + [3000]
    cache, table, n = paged(lens, 2, 64, 16, BF16)
    q = rand((len(lens), 4, 64), 5, BF16, 2.0)
    want, bound = R.step(q, cache.k, cache.v, table, n)
    within("step many", A.attention_step(q, cache, table, n), want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 41])
@pytest.mark.parametrize("most", [256, 257])
def test_step_many_short_sequences(most, window, dtype):
    """Enough sequences of eight steps or fewer for a block to take a whole one, and of nine."""
    lens = [(i * 37) % (most + 1) for i in range(260)]
    cache, table, n = paged(lens, 2, 72, 16, dtype)
    q = rand((len(lens), 6, 72), 5, dtype, 2.0)
    want, bound = R.step(q, cache.k, cache.v, table, n, window)
    within("step short", A.attention_step(q, cache, table, n, window=window), want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [4, 60])
def test_step_wide_groups(width, dtype):
    """Groups of more heads than a tile has columns, with blocks of whole sequences and without."""
    lens = [0, 1, 40, 64]
    cache, table, n = paged(lens, 2, 40, 16, dtype, width=width)
    q = rand((len(lens), 80, 40), 5, dtype, 2.0)
    want, bound = R.step(q, cache.k, cache.v, table, n)
    within("step wide", A.attention_step(q, cache, table, n), want, bound)


def test_step_most_sequences():
    """65535 sequences of one key each, of so many key heads that a thread for each channel of
    each is more than 2^32 threads: the answer is that key's value."""
    batch, hk, dh = 65535, 130, 8
    k, v = rand((1, hk, 64, dh), 1, BF16), rand((1, hk, 64, dh), 2, BF16)
    table = torch.zeros(batch, 5, dtype=torch.int32, device=DEV)
    n = torch.ones(batch, dtype=torch.int32, device=DEV)
    n[7] = 0
    q = torch.randn(batch, hk, dh, device=DEV).to(BF16)
    o = A.attention_step(q, A.KVCache(k, v), table, n)
    want = v[:, :, 0].expand(batch, hk, dh).clone()
    want[7] = 0
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_pages_that_are_none(dtype):
    """Keys of pages outside the cache are not there; lengths outside the table are cut to it."""
    lens = [100, 64, 1000, 30]
    cache, table, n = paged(lens, 2, 64, 16, dtype)
    q = rand((4, 4, 64), 5, dtype, 2.0)
    table[0, 2], table[1, :], table[2, 5], table[2, 20] = -1, 10 ** 6, cache.pages, -7
    want, bound = R.step(q, cache.k, cache.v, table, n)
    assert (want[1] == 0).all()
    within("step no pages", A.attention_step(q, cache, table, n), want, bound)
    far = torch.tensor([100, 2 ** 31 - 1, 1000, -3], dtype=torch.int32, device=DEV)
    o = A.attention_step(q, cache, table, far)
    assert torch.equal(o[0], A.attention_step(q, cache, table, n)[0]) and (o[1] == 0).all() and (o[3] == 0).all()


def test_step_at_the_last_place_that_32_bits_count():
    """Lengths to 2^31 - 2 through a table that names the same pages again and again."""
    page, width, dh = 49981, 42966, 64      # their product is 2^31 - 2
    cache = A.KVCache(rand((3, 1, page, dh), 1, BF16), rand((3, 1, page, dh), 2, BF16))
    table = (torch.arange(width, device=DEV) % 3).to(torch.int32)[None].repeat(2, 1)
    n = torch.tensor([page * width, 2 ** 31 - 40], dtype=torch.int32, device=DEV)
    q = rand((2, 4, dh), 3, BF16, 2.0)
    for window in (1, 31, 1000):
        want, bound = R.step(q, cache.k, cache.v, table, n, window)
        within("step far", A.attention_step(q, cache, table, n, window=window), want, bound)


def test_step_lse():
    """The C entry's log sums."""
    lens, hq, hk, dh, page, _ = STEPS[3]
    cache, table, n = paged(lens, hk, dh, page, F32)
    q = rand((len(lens), hq, dh), 5, F32, 2.0)
    o, lse = torch.empty_like(q), torch.empty((len(lens), hq), device=DEV)
    desc, tab = A.StepDesc(hq, 0, dh ** -0.5), cache.table(table)
    need = A.ipttt_attention_step_workspace_bytes(desc, cache.desc, tab)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    A.ipttt_attention_step(desc, A._heads("q", q, q.shape, F32, q.device), cache.desc, tab, n,
                           A._heads("o", o, q.shape, F32, q.device), lse, ws, need)
    assert torch.equal(o, A.attention_step(q, cache, table, n))
    for b, m in enumerate(lens):
        if m == 0:
            assert (lse[b] == -math.inf).all()
            continue
        at = torch.arange(m, device=DEV)
        page_of = table[b].long()[at // page]
        for h in range(hq):
            k = cache.k[page_of, h // (hq // hk), at % page].double()
            want = torch.logsumexp(q[b, h].double() @ k.T * dh ** -0.5, 0)
            assert abs(lse[b, h].item() - want.item()) <= 2e-5


# ---- together -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 40])
def test_prefill_then_decode(window, dtype):
    """Prompts of different lengths prefilled and appended, then decoded token by token through
    the cache, against attention over the whole sequences."""
    hq, hk, dh, page = 4, 2, 64, 16
    lens, more = [70, 1, 33], 40
    op, *_ = head_op(hq, hk, dh, dh, False, "qk", dtype)
    whole = [rand((m + more, (hq + 2 * hk), dh), 50 + i, dtype) for i, m in enumerate(lens)]
    width = -(-(max(lens) + more) // page)
    cache = A.KVCache.empty(3 * width, hk, page, dh, dtype, DEV)
    table = torch.randperm(3 * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(3, width).to(DEV)

    def parts(x):
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]

    packed = torch.cat([w[:m] for w, m in zip(whole, lens)])
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).to(DEV)
    seqs = torch.cat([torch.full((m,), i, dtype=torch.int32) for i, m in enumerate(lens)]).to(DEV)
    q, k, v = parts(packed)
    qr = op.append(q, k, v, pos, cache, table, seqs)
    _, kr = op.forward(q, k, pos)
    o, _ = A.attention_forward(qr, kr, v, offsets=offsets(lens), window=window)
    # the oracle: whole sequences
    wants = []
    for w in whole:
        q, k, v = parts(w)
        qr, kr = op.forward(q, k, torch.arange(w.shape[0], dtype=torch.int32, device=DEV))
        wants.append(R.attention(qr, kr, v, [w.shape[0]], [w.shape[0]], True, window))
    at = 0
    for i, m in enumerate(lens):
        within("prefill", o[at:at + m], wants[i][0][:m], wants[i][2][:m])
        at += m
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for t in range(more):
        new = torch.stack([w[m + t] for w, m in zip(whole, lens)])
        q, k, v = parts(new)
        qr = op.append(q, k, v, n, cache, table)
        n += 1
        o = A.attention_step(qr, cache, table, n, window=window)
        for i, m in enumerate(lens):
            within("decode", o[i], wants[i][0][m + t], wants[i][2][m + t])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_results_repeat(dtype):
    """Bit for bit, whatever the memory held that outputs and workspace come from."""
    q, k, v, dy, lq, lk, how = prompt(([700, 1, 90], None, 4, 2, 128, True, 0), dtype)
    cache, table, n = paged([5000, 70], 2, 128, 16, dtype)
    op, *_ = head_op(4, 2, 128, 128, False, "qk", dtype)
    pos = torch.arange(q.shape[0], dtype=torch.int32, device=DEV)

    def all_of():
        o, lse = A.attention_forward(q, k, v, **how)
        h = op.backward(q, k, pos, dy, k)
        return [o, lse, *A.attention_backward(q, k, v, o, lse, dy, **how).values(), *op.forward(q, k, pos),
                *h.values(), A.attention_step(q[:2], cache, table, n)]

    want = all_of()
    for _ in range(3):
        junk = [torch.full((1 << s,), 255, dtype=torch.uint8, device=DEV) for s in range(8, 25) for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(all_of(), want))

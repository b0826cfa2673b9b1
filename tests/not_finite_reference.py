"""Attention in 64 bits where some of what it reads is not finite: the sums go over what a query
sees and nothing else, term by term, so that a hidden term adds no 0 x infinity. Helpers only;
no tests here.

`agree` holds a result to the formula's class: where that is finite the result is within its
bound (counted as in attention_reference), where it is NaN the result is NaN, and where it is an
infinity the result is no finite number (it may be NaN)."""
from __future__ import annotations

import torch

from attention_reference import E32, half_step, w64


def _rounding(dtype):
    return half_step(dtype), half_step(torch.bfloat16) if dtype is torch.bfloat16 else 0.0


def _sum(ok, terms, dim):
    return torch.where(ok, terms, 0.0).sum(dim)


def forward(q, k, v, ok, scale, dtype):
    """(o, lse, bound of o, bound of lse) of one head: q [n, dh], k and v [m, dh], ok [n, m]."""
    out, weight = _rounding(dtype)
    q, k, v = w64(q), w64(k), w64(v)
    a = (q[:, None] * k[None]).sum(-1) * scale
    live = ok.any(1)
    a = torch.where(ok, a, -torch.inf)
    lse = torch.logsumexp(a, 1)
    p = torch.where(ok, torch.exp(a - lse[:, None]), 0.0)
    o = torch.where(live[:, None], _sum(ok[..., None], p[..., None] * v[None], 1), 0.0)
    size = (q.abs()[:, None] * k.abs()[None]).sum(-1) * abs(scale)
    size = torch.where(ok & torch.isfinite(a), size, 0.0).amax(1)
    score = E32 * ((q.shape[1] + 4) * size + 8)
    fp32 = 2 * score + E32 * (ok.sum(1) + 16)
    mass = _sum(ok[..., None], p[..., None] * v.abs()[None], 1)
    return (o, lse, (weight + fp32[:, None]) * mass * 1.02 + out * o.abs() * 1.02,
            fp32 + E32 * 4 * lse.abs().nan_to_num(0, 0, 0))


def backward(q, k, v, dy, o, lse, ok, scale, dtype):
    """{dq, dk, dv: (value, bound before the rounding to the output's type)} of one head, from the
    forward's results."""
    out, weight = _rounding(dtype)
    q, k, v, dy, o, lse = (w64(t) for t in (q, k, v, dy, o, lse))
    a = (q[:, None] * k[None]).sum(-1) * scale
    p = torch.where(ok, torch.exp(a - lse[:, None]), 0.0)
    dp = (dy[:, None] * v[None]).sum(-1)
    delta = (dy * o).sum(1, keepdim=True)
    ds = torch.where(ok, p * (dp - delta) * scale, 0.0)
    dh = q.shape[1]
    size = (q.abs()[:, None] * k.abs()[None]).sum(-1) * abs(scale)
    size = torch.where(torch.isfinite(a), size, 0.0)
    perr = p * E32 * ((dh + 4) * size + 8 + 2 * lse[:, None].abs().nan_to_num(0, 0, 0))
    dperr = E32 * (dh + 8) * ((dy.abs()[:, None] * v.abs()[None]).sum(-1) + (dy * o).abs().sum(1, keepdim=True))
    dserr = abs(scale) * (perr * (dp - delta).abs() + p * dperr) + weight * ds.abs() + E32 * 4096 * ds.abs()
    perr = perr + weight * p + E32 * 4096 * p
    ok = ok[..., None]

    def both(w, err, x, dim):
        x = x[None] if dim == 1 else x[:, None]
        return _sum(ok, w[..., None] * x, dim), _sum(ok, err[..., None] * x.abs(), dim)

    return {"dq": both(ds, dserr, k, 1), "dk": both(ds, dserr, q, 0), "dv": both(p, perr, dy, 0)}


def agree(name, got, want, bound):
    got = got.double()
    finite, nan = torch.isfinite(want), torch.isnan(want)
    wrong = torch.where(finite, ~((got - want).abs() <= bound + 1e-37), torch.where(nan, ~torch.isnan(got), torch.isfinite(got)))
    if wrong.any():
        at = tuple(wrong.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(wrong.sum())} of {wrong.numel()} wrong, the first at {at}: "
                             f"{got[at].item()}, the formula {want[at].item()}")

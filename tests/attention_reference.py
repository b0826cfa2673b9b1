"""The attention operators in 64 bits, written from their formulas, and bounds of what
rounding may do to them. Helpers only; no tests here.

A bound counts the roundings of the operator it is for, worst case by worst case: one to
the output's type (half a step, relative), one to bf16 of each weight p or gradient ds that
enters a product, and the fp32 arithmetic in between."""
from __future__ import annotations

import math

import torch

E32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def w64(t):
    return t.detach().to(torch.float64)


# ---- head norm --------------------------------------------------------------------------


def rotate(x, pos, inv_freq, interleaved, back=False):
    """[n, heads, dh] by pos [n] * inv_freq, channel pair by channel pair."""
    r2 = inv_freq.numel()
    y = x.clone()
    for i in range(r2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r2)
        angle = pos.double() * float(inv_freq[i]) * (-1 if back else 1)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def head_forward(x, gamma, pos, inv_freq, eps, interleaved):
    x = w64(x)
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w64(gamma)
    return rotate(x, pos, inv_freq, interleaved)


def head_backward(x, gamma, pos, inv_freq, eps, interleaved, dy):
    """(dx, dgamma or None)."""
    x, g = w64(x), rotate(w64(dy), pos, inv_freq, interleaved, back=True)
    if gamma is None:
        return g, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    w = g * w64(gamma)
    return r * (w - x * r * (w * x * r).mean(-1, keepdim=True)), (g * x * r).sum((0, 1))


# ---- attention --------------------------------------------------------------------------


def seen(lq, lk, causal, window, device):
    """[lq, lk]: which keys a query sees."""
    last = torch.arange(lq, device=device)[:, None] + lk - lq
    j = torch.arange(lk, device=device)[None]
    if not causal:
        return torch.ones((lq, lk), dtype=torch.bool, device=device)
    ok = j <= last
    return ok & (j > last - window) if window else ok


def sequences(lq, lk):
    at = k_at = 0
    for m, n in zip(lq, lk):
        yield slice(at, at + m), slice(k_at, k_at + n)
        at, k_at = at + m, k_at + n


def attention(q, k, v, lq, lk, causal=True, window=0, scale=None):
    """(o, lse, bound of o's error, bound of lse's) for packed sequences of these lengths; what
    lies behind them is zero."""
    n, hq, dh = q.shape
    group = hq // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    out = half_step(q.dtype)
    weight = half_step(torch.bfloat16) if q.dtype is torch.bfloat16 else 0.0
    o, bound = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    lse_bound = torch.zeros_like(lse)
    for rows, keys in sequences(lq, lk):
        if rows.stop == rows.start or keys.stop == keys.start:
            continue
        ok = seen(rows.stop - rows.start, keys.stop - keys.start, causal, window, q.device)
        live = ok.any(1)
        for h in range(hq):
            qq, kk, vv = w64(q[rows, h]), w64(k[keys, h // group]), w64(v[keys, h // group])
            a = torch.where(ok, qq @ kk.T * scale, -math.inf)
            top = torch.where(live, a.amax(1), 0.0)[:, None]
            p = torch.exp(a - top)
            total = p.sum(1, keepdim=True).clamp_min(1e-300)
            p = p / total
            o[rows, h] = p @ vv
            lse[h, rows] = torch.where(live, (top + torch.log(total))[:, 0], -math.inf)
            # a score: dh products and sums, the factor, its difference from the maximum
            size = torch.where(ok, qq.abs() @ kk.abs().T * abs(scale), 0.0).amax(1)
            score = E32 * ((dh + 4) * size + 8)
            keys_n = ok.sum(1).double()
            mass = p @ vv.abs()
            fp32 = (2 * score + E32 * (keys_n.clamp_max(4096) + 16))[:, None]
            bound[rows, h] = ((weight + fp32) * mass * 1.02 + out * o[rows, h].abs() * 1.02)
            lse_bound[h, rows] = 2 * score + E32 * (keys_n.clamp_max(4096) + 16) + E32 * 4 * lse[h, rows].nan_to_num(0, 0, 0).abs()
    return o, lse, bound, lse_bound


def attention_backward(q, k, v, o, lse, dy, lq, lk, causal=True, window=0, scale=None):
    """({dq, dk, dv}, their bounds) from the forward's results."""
    n, hq, dh = q.shape
    group = hq // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    out = half_step(q.dtype)
    weight = half_step(torch.bfloat16) if q.dtype is torch.bfloat16 else 0.0
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=t.device)  # noqa: E731
    got, bound = ({"dq": z(q), "dk": z(k), "dv": z(k)} for _ in range(2))
    for rows, keys in sequences(lq, lk):
        if rows.stop == rows.start or keys.stop == keys.start:
            continue
        ok = seen(rows.stop - rows.start, keys.stop - keys.start, causal, window, q.device)
        for h in range(hq):
            g = h // group
            qq, kk, vv, yy = w64(q[rows, h]), w64(k[keys, g]), w64(v[keys, g]), w64(dy[rows, h])
            p = torch.where(ok, torch.exp(qq @ kk.T * scale - w64(lse[h, rows])[:, None]), 0.0)
            delta = (yy * w64(o[rows, h])).sum(1, keepdim=True)
            dp = yy @ vv.T
            ds = p * (dp - delta) * scale
            got["dq"][rows, h] = ds @ kk
            got["dk"][keys, g] += ds.T @ qq
            got["dv"][keys, g] += p.T @ yy
            # fp32: the score (with lse's own error left out: it is an input), dp and delta
            size = torch.where(ok, qq.abs() @ kk.abs().T * abs(scale), 0.0)
            perr = p * E32 * ((dh + 4) * size + 8 + 2 * w64(lse[h, rows])[:, None].nan_to_num(0, 0, 0).abs())
            dperr = E32 * (dh + 8) * (yy.abs() @ vv.abs().T + (yy.abs() * w64(o[rows, h]).abs()).sum(1, keepdim=True))
            dserr = abs(scale) * (perr * (dp - delta).abs() + p * dperr) + weight * ds.abs()
            perr = perr + weight * p
            acc = E32 * 4096
            bound["dq"][rows, h] = dserr @ kk.abs() + acc * (ds.abs() @ kk.abs())
            bound["dk"][keys, g] += dserr.T @ qq.abs() + acc * (ds.abs().T @ qq.abs())
            bound["dv"][keys, g] += perr.T @ yy.abs() + acc * (p.T @ yy.abs())
    for x in got:
        bound[x] = bound[x] * 1.05 + out * got[x].abs() * 1.02
    return got, bound


def gathered(pages, table, page_size, length, head, n_pages):
    """(rows, which of them are there) of one sequence's head from a paged cache."""
    rows, there = [], []
    for t in range(length):
        p = int(table[t // page_size])
        ok = 0 <= p < n_pages
        there.append(ok)
        rows.append(w64(pages[p if ok else 0, head, t % page_size]))
    return torch.stack(rows), torch.tensor(there, device=pages.device)


def step(q, k_pages, v_pages, table, lens, window=0, scale=None):
    """(o, bound of its error) for one new token a sequence."""
    n, hq, dh = q.shape
    pages, hk, ps, _ = k_pages.shape
    scale = dh ** -0.5 if scale is None else scale
    weight = half_step(torch.bfloat16) if q.dtype is torch.bfloat16 else 0.0
    o, bound = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    tab = table.tolist()
    for b in range(n):
        m = min(max(int(lens[b]), 0), table.shape[1] * ps)
        lo = max(0, m - window) if window else 0
        if m == 0:
            continue
        at = torch.arange(lo, m, device=q.device)
        page = torch.tensor(tab[b], device=q.device)[at // ps]
        ok = (page >= 0) & (page < pages)
        at, page = at[ok], page[ok]
        if at.numel() == 0:
            continue
        for h in range(hk):
            kk, vv = w64(k_pages[page, h, at % ps]), w64(v_pages[page, h, at % ps])
            hs = slice(h * (hq // hk), (h + 1) * (hq // hk))
            qq = w64(q[b, hs])
            p = torch.softmax(qq @ kk.T * scale, 1)
            o[b, hs] = p @ vv
            size = (qq.abs() @ kk.abs().T * abs(scale)).amax(1, keepdim=True)
            fp32 = E32 * (2 * (dh + 4) * size + 4096 + 32)
            bound[b, hs] = (weight + fp32) * (p @ vv.abs()) * 1.02 + half_step(q.dtype) * o[b, hs].abs() * 1.02
    return o, bound

"""The block operators in 64 bits on the CPU, written from their formulas, token by
token and row by row where that is the definition. Helpers only; no tests here."""
from __future__ import annotations

import torch


def d64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def norm_forward(x, r, gamma, beta, eps):
    h = d64(x) if r is None else d64(x) + d64(r)
    mean = h.mean(-1, keepdim=True)
    c = h - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    y = c * rstd
    if gamma is not None:
        y = y * d64(gamma)
    if beta is not None:
        y = y + d64(beta)
    return y, h, mean[..., 0], rstd[..., 0]


def norm_backward(h, mean, rstd, gamma, dy, dh):
    h, dy = d64(h), d64(dy)
    xh = (h - d64(mean)[:, None]) * d64(rstd)[:, None]
    q = dy if gamma is None else dy * d64(gamma)
    dx = (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True)) * d64(rstd)[:, None]
    if dh is not None:
        dx = dx + d64(dh)
    return dx, (dy * xh).sum(0), dy.sum(0)


def recurrence(g, v, h0, starts, lens):
    """(h, h_last), one token after another."""
    g, v = d64(g), d64(v)
    n, length, d = g.shape
    out = torch.zeros_like(g)
    last = torch.zeros((n, d), dtype=torch.float64)
    for i in range(n):
        s = torch.zeros(d, dtype=torch.float64) if h0 is None else d64(h0[i]).clone()
        m = length if lens is None else min(max(int(lens[i]), 0), length)
        for t in range(m):
            if starts is not None and int(starts[i, t]):
                s = torch.zeros_like(s)
            f = torch.sigmoid(g[i, t])
            s = f * s + torch.sigmoid(-g[i, t]) * v[i, t]
            out[i, t] = s
        last[i] = s
    return out, last


def recurrence_backward(g, v, h, dh, h0, dh_last, starts, lens):
    """(dg, dv, dh0) from the saved h, last token first."""
    g, v, h, dh = d64(g), d64(v), d64(h), d64(dh)
    n, length, d = g.shape
    dg, dv = torch.zeros_like(g), torch.zeros_like(g)
    dh0 = torch.zeros((n, d), dtype=torch.float64)
    for i in range(n):
        s = torch.zeros(d, dtype=torch.float64) if dh_last is None else d64(dh_last[i]).clone()
        m = length if lens is None else min(max(int(lens[i]), 0), length)
        for t in range(m - 1, -1, -1):
            cut = starts is not None and int(starts[i, t])
            f, k = torch.sigmoid(g[i, t]), torch.sigmoid(-g[i, t])
            if cut:
                prev = torch.zeros_like(s)
            elif t:
                prev = h[i, t - 1]
            else:
                prev = torch.zeros_like(s) if h0 is None else d64(h0[i])
            delta = dh[i, t] + s
            dv[i, t] = k * delta
            dg[i, t] = delta * (prev - v[i, t]) * f * k
            s = torch.zeros_like(s) if cut else f * delta
        dh0[i] = s
    return dg, dv, dh0


def ff_forward(x, wg, wu, wd):
    x = d64(x)
    a, u = x @ d64(wg).T, x @ d64(wu).T
    return (a * torch.sigmoid(a) * u) @ d64(wd).T, a, u


def ff_backward(x, wg, wu, wd, dy):
    """(dx, dw_gate, dw_up, dw_down) by the chain rule."""
    _, a, u = ff_forward(x, wg, wu, wd)
    x, dy = d64(x), d64(dy)
    s = torch.sigmoid(a)
    z, dz = a * s * u, dy @ d64(wd)
    da, du = dz * u * (s + a * s * (1 - s)), dz * a * s
    return da @ d64(wg) + du @ d64(wu), da.T @ x, du.T @ x, dy.T @ z

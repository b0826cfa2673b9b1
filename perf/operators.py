"""Cases of the block operators around the fast-weight layer: layer norm, the gated linear recurrence
and the gated feed-forward block, each with its backward pass and its form for single tokens.

`run` computes a case in plain torch operations where `own` is false and through
chunked_weight_mlp_amd.block where it is true. Shapes are the repository's own layer shapes (the
4B-shaped layer, d 2560 and d_ff 9728, and the 1.5B-shaped one, d 2048 and d_ff 8192) and odd ones.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # --- layer norm ---
        # decoding: the residual add and norm in front of a layer, eight sequences, one token each
        dict(name="norm_decode", op="norm", way="forward", dtype="bf16", n=8, d=2560, res=True),
        # prefill of a 32k document: residual add and norm in front of the 4B-shaped layer
        dict(name="norm_prefill", op="norm", way="forward", dtype="bf16", n=32768, d=2560, res=True),
        # training the 1.5B-shaped layer on 8 x 16k tokens: gradient of a norm inside a residual block
        dict(name="norm_train", op="norm", way="backward", dtype="bf16", n=131072, d=2048, res=True),
        # a small fp32 model of odd width, ragged row count
        dict(name="norm_odd_f32", op="norm", way="backward", dtype="f32", n=1021, d=1543, res=False),
        # --- gated linear recurrence ---
        # decoding: one token for each of 32 sequences
        dict(name="mix_decode", op="mix", way="step", dtype="bf16", n=32, len=1, d=2560, fused=True,
             starts=False, ragged=False),
        # prefill of one 128k document, gate and value from one fused projection
        dict(name="mix_prefill_128k", op="mix", way="forward", dtype="bf16", n=1, len=131072, d=2560,
             fused=True, starts=False, ragged=False),
        # training on 8 x 16k tokens of packed documents
        dict(name="mix_train_packed", op="mix", way="backward", dtype="bf16", n=8, len=16384, d=2048,
             fused=True, starts=True, ragged=False),
        # a batch of prompts of different lengths, fp32, odd sizes
        dict(name="mix_ragged_f32", op="mix", way="forward", dtype="f32", n=5, len=1237, d=331,
             fused=False, starts=True, ragged=True),
        # --- gated feed-forward block ---
        # decoding a single sequence: every weight is read for one token
        dict(name="ff_token", op="ff", way="forward", dtype="bf16", n=1, d=2560, f=9728, pad=0),
        # prefill of a slab of tokens through the 4B-shaped block
        dict(name="ff_prefill", op="ff", way="forward", dtype="bf16", n=16384, d=2560, f=9728, pad=0),
        # a training step's tokens through the 1.5B-shaped block, forward and backward
        dict(name="ff_train", op="ff", way="train", dtype="bf16", n=8192, d=2048, f=8192, pad=0),
        # a small fp32 block of odd sizes, trained on rows that are a slice of a wider buffer
        dict(name="ff_odd_f32", op="ff", way="train", dtype="f32", n=333, d=250, f=671, pad=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly multiples of 64, as models have, some of 8, some of no kind."""
    w = _log(rng, lo, hi)
    k = rng.random()
    if k < 0.55:
        return max(64, w // 64 * 64)
    if k < 0.75:
        return max(8, w // 8 * 8)
    return w


def draw(rng):
    op = rng.choice(["norm", "mix", "ff"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "norm":
        d = _width(rng, 32, 8192)
        most = min(131072, 131072 * 2048 // d)
        return dict(op=op, way=rng.choice(["forward", "backward"]), dtype=dtype,
                    n=_log(rng, 1, most), d=d, res=rng.random() < 0.7)
    if op == "mix":
        way = rng.choice(["step", "forward", "forward", "backward", "backward"])
        d = _width(rng, 16, 2560)
        n = _log(rng, 1, 128 if way == "step" else 16)
        most = 131072 * 2560 // (n * d * (2 if dtype == "f32" or way == "backward" else 1))
        return dict(op=op, way=way, dtype=dtype, n=n,
                    len=1 if way == "step" else _log(rng, 1, min(131072, most)), d=d,
                    fused=rng.random() < 0.5, starts=way != "step" and rng.random() < 0.5,
                    ragged=way != "step" and rng.random() < 0.3)
    way = rng.choice(["forward", "forward", "train"])
    return dict(op=op, way=way, dtype=dtype, n=_log(rng, 1, 8192), d=_width(rng, 32, 2048),
                f=_width(rng, 64, 8192), pad=rng.choice([0, 0, 8, 3]))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g, t = _gen(seed), TYPES[case["dtype"]]
    s = dict(case=case)
    n, d = case["n"], case["d"]
    if case["op"] == "norm":
        # the residual stream: a few channels much larger than the others
        scale = torch.where(torch.rand(d, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s["gamma"] = (1.0 + _normal(g, (d,), torch.float32, 0.2)).to(t)
        s["beta"] = _normal(g, (d,), t, 0.1)
        s["x"] = (_normal(g, (n, d), torch.float32) * scale + 0.1).to(t)
        s["res"] = _normal(g, (n, d), t) if case["res"] else None
        if case["way"] == "backward":
            s["dy"] = _normal(g, (n, d), t)
            s["dh"] = s.pop("res")
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        if own:
            from chunked_weight_mlp_amd import block
            s["norm"] = block.Norm(s["gamma"], s["beta"], eps=EPS)
        return s
    if case["op"] == "mix":
        length = case["len"]
        both = torch.empty((n, length, 2 * d), dtype=t, device=DEV)
        # gates mostly remember (trained forget gates sit near one), a few forget at once
        for i in range(n):
            both[i, :, :d] = _normal(g, (length, d), torch.float32, 2.0) + 3.0
            both[i, :, d:] = _normal(g, (length, d), t)
        s["starts"] = s["lens"] = None
        if case["starts"]:
            s["starts"] = (torch.rand((n, length), generator=g, device=DEV) < 1 / 1500).to(torch.uint8)
        if case["ragged"]:
            s["lens"] = torch.randint(0, length + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
            past = torch.arange(length, device=DEV)[None, :] >= s["lens"][:, None]
            both[past] = float("nan")  # nothing is written there
        gate, value = both[..., :d], both[..., d:]
        if not case["fused"]:
            gate, value = gate.contiguous(), value.contiguous()
        s["g"], s["v"] = gate, value
        s["h0"] = _normal(g, (n, d), torch.float32, 0.3)
        if case["way"] == "backward":
            h, _ = _plain_mix(s)
            s["h"] = h
            s["dh"] = _normal(g, (n, length, d), t)
            s["dh_last"] = _normal(g, (n, d), torch.float32)
        return s
    f, pad = case["f"], case["pad"]
    s["x"] = _normal(g, (n, d + pad), t)[:, :d]
    s["w_gate"] = _normal(g, (f, d), t, d ** -0.5)
    s["w_up"] = _normal(g, (f, d), t, d ** -0.5)
    s["w_down"] = _normal(g, (d, f), t, f ** -0.5)
    if case["way"] == "train":
        s["dy"] = _normal(g, (n, d + pad), t)[:, :d]
    if own:
        from chunked_weight_mlp_amd import block
        s["ff"] = block.FeedForward(s["w_gate"], s["w_up"], s["w_down"])
    return s


# ---- plain forms -----------------------------------------------------------------------------


def _plain_norm(s):
    t = s["x"].dtype
    if s["case"]["way"] == "forward":
        h = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
        mean = h.mean(1)
        c = h - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(1) + EPS)
        y = c * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(t), "h": h.to(t), "mean": mean, "rstd": rstd}
    h, dy = s["x"].float(), s["dy"].float()
    xh = (h - s["mean"][:, None]) * s["rstd"][:, None]
    gd = dy * s["gamma"].float()
    dx = (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(t), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, h_{-1} = 0, by doubling (both are overwritten)."""
    k, length = 1, a.shape[1]
    while k < length:
        b[:, k:] = torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _mix_parts(s):
    """f, 1 - f (both 0 past a row's length), f with the cut at document starts, the valid places."""
    g = s["g"].float()
    live = None
    if s["lens"] is not None:
        live = (torch.arange(g.shape[1], device=g.device)[None, :] < s["lens"][:, None])[..., None]
        g = torch.where(live, g, torch.zeros_like(g))
    f, i = torch.sigmoid(g), torch.sigmoid(-g)
    cut = f if s["starts"] is None else torch.where((s["starts"] != 0)[..., None], torch.zeros_like(f), f)
    return f, i, cut, live


def _plain_mix(s):
    f, i, cut, live = _mix_parts(s)
    v = s["v"].float() if live is None else torch.where(live, s["v"].float(), torch.zeros_like(f))
    n, length, d = f.shape
    b = i * v
    b[:, 0] += cut[:, 0] * s["h0"]
    h = _scan(cut.clone(), b)
    if live is None:
        return h.to(s["g"].dtype), h[:, -1].clone()
    last = torch.cat([s["h0"][:, None], h], 1)
    last = torch.gather(last, 1, s["lens"].long()[:, None, None].expand(n, 1, d))[:, 0]
    return torch.where(live, h, torch.zeros_like(h)).to(s["g"].dtype), last


def _plain_mix_backward(s):
    f, i, cut, live = _mix_parts(s)
    n, length, d = f.shape
    if live is not None:
        v, h, dh = (torch.where(live, s[k].float(), torch.zeros_like(f)) for k in ("v", "h", "dh"))
    else:
        v, h, dh = s["v"].float(), s["h"].float(), s["dh"].float().clone()
    prev = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    if s["starts"] is not None:
        prev = torch.where((s["starts"] != 0)[..., None], torch.zeros_like(prev), prev)
    # delta_t = dh_t + cut_{t+1} delta_{t+1}; dh_last joins at each row's last token
    if live is None:
        dh[:, -1] += s["dh_last"]
    else:
        row = torch.arange(n, device=f.device)
        at = (s["lens"].long() - 1).clamp_min(0)
        dh[row, at] += torch.where((s["lens"] > 0)[:, None], s["dh_last"], torch.zeros_like(s["dh_last"]))
    nxt = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    if live is not None:
        nxt = nxt * torch.cat([live[:, 1:], torch.zeros_like(live[:, :1])], 1)
    delta = _scan(nxt.flip(1), dh.flip(1)).flip(1)
    dv, dg = i * delta, delta * (prev - v) * f * i
    dh0 = cut[:, 0] * delta[:, 0]
    if live is not None:
        dv, dg = (torch.where(live, x, torch.zeros_like(x)) for x in (dv, dg))
        dh0 = torch.where((s["lens"] > 0)[:, None], dh0, s["dh_last"])
    t = s["g"].dtype
    return {"dg": dg.to(t), "dv": dv.to(t), "dh0": dh0}


def _plain_ff(s):
    t = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    a, u = x @ wg.t(), x @ wu.t()
    sg = torch.sigmoid(a)
    z = a * sg * u
    out = {"y": (z @ wd.t()).to(t)}
    if s["case"]["way"] == "train":
        dy = s["dy"].float()
        dz = dy @ wd
        da, du = dz * u * sg * (1 + a * (1 - sg)), dz * a * sg
        out["dx"] = (da @ wg + du @ wu).to(t)
        out["dw_gate"] = (da.t() @ x).to(t)
        out["dw_up"] = (du.t() @ x).to(t)
        out["dw_down"] = (dy.t() @ z).to(t)
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "norm":
            return _plain_norm(s)
        if case["op"] == "ff":
            return _plain_ff(s)
        if case["way"] == "backward":
            return _plain_mix_backward(s)
        h, last = _plain_mix(s)
        return {"h": h, "h_last": last}
    from chunked_weight_mlp_amd import block
    if case["op"] == "norm":
        if case["way"] == "forward":
            y, h, mean, rstd = s["norm"].forward(s["x"], s["res"])
            return {"y": y, "h": h, "mean": mean, "rstd": rstd}
        return s["norm"].backward(s["x"], s["mean"], s["rstd"], s["dy"], s["dh"])
    if case["op"] == "mix":
        if case["way"] == "step":
            h, last = block.recurrence_step(s["g"][:, 0], s["v"][:, 0], s["h0"])
            return {"h": h[:, None], "h_last": last}
        if case["way"] == "forward":
            h, last = block.recurrence_forward(s["g"], s["v"], h0=s["h0"], starts=s["starts"],
                                               lens=s["lens"])
            return {"h": h, "h_last": last}
        return block.recurrence_backward(s["g"], s["v"], s["h"], s["dh"], h0=s["h0"],
                                         dh_last=s["dh_last"], starts=s["starts"], lens=s["lens"])
    if case["way"] == "forward":
        return {"y": s["ff"].forward(s["x"])}
    y, a, u = s["ff"].forward(s["x"], save=True)
    return {"y": y, **s["ff"].backward(s["x"], a, u, s["dy"])}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n, d = case["n"], case["d"]
    if case["op"] == "norm":
        # forward: x, r -> y, h; backward: h, dy, dh -> dx
        rows = (4 if case["res"] else 2) if case["way"] == "forward" else (4 if case["res"] else 3)
        return {"bytes": rows * n * d * e + 8 * n + 4 * d * e, "flops": 10 * n * d}
    if case["op"] == "mix":
        el = n * case["len"] * d
        # forward: g, v -> h; backward: g, v, h, dh -> dg, dv
        return {"bytes": (6 if case["way"] == "backward" else 3) * el * e + 8 * n * d, "flops": 10 * el}
    f = case["f"]
    if case["way"] == "forward":
        return {"bytes": (3 * d * f + 2 * n * d) * e, "flops": 6 * n * d * f}
    return {"bytes": (6 * d * f + 4 * n * d) * e, "flops": 18 * n * d * f}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    w = lambda k: s[k].double()  # noqa: E731
    if case["op"] == "norm":
        if case["way"] == "forward":
            h = w("x") + (0 if s["res"] is None else w("res"))
            var, mean = torch.var_mean(h, 1, correction=0)
            rstd = 1 / (var + EPS).sqrt()
            y = torch.addcmul(w("beta"), (h - mean[:, None]) * rstd[:, None], w("gamma"))
            return {"y": y, "h": h, "mean": mean, "rstd": rstd}
        # y = xh gamma + beta with xh = (h - mean) rstd: the chain rule through the given statistics
        xh = (w("x") - w("mean")[:, None]) * w("rstd")[:, None]
        dxh = w("dy") * w("gamma")
        d = case["d"]
        dx = w("rstd")[:, None] / d * (d * dxh - dxh.sum(1, True) - xh * (dxh * xh).sum(1, True))
        if s["dh"] is not None:
            dx = dx + w("dh")
        return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", w("dy"), xh), "dbeta": w("dy").sum(0)}
    if case["op"] == "mix":
        return _exact_mix(s, case)
    x, wg, wu, wd = w("x"), w("w_gate"), w("w_up"), w("w_down")
    a, u = x.mm(wg.T), x.mm(wu.T)
    gate = a / (1 + torch.exp(-a))
    out = {"y": (gate * u).mm(wd.T)}
    if case["way"] == "train":
        dz = w("dy").mm(wd)
        out["dw_down"] = w("dy").T.mm(gate * u)
        du = dz * gate
        # SiLU'(a) = s + a s (1 - s), s = 1 / (1 + e^-a)
        sg = 1 / (1 + torch.exp(-a))
        da = dz * u * (sg + gate * (1 - sg))
        out["dx"] = da.mm(wg) + du.mm(wu)
        out["dw_gate"], out["dw_up"] = da.T.mm(x), du.T.mm(x)
    return out


def _exact_mix(s, case):
    """Token by token, as the recurrence is written."""
    n, length, d = s["g"].shape
    lens = [length] * n if s["lens"] is None else s["lens"].tolist()
    live = torch.tensor([[t < m for t in range(length)] for m in lens], device=DEV)[..., None]
    g = s["g"].double().masked_fill(~live, 0)
    v = s["v"].double().masked_fill(~live, 0)
    f, i = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    go = torch.ones((n, length, 1), dtype=torch.float64, device=DEV)
    if s["starts"] is not None:
        go = (s["starts"] == 0).double()[..., None]
    state = s["h0"].double()
    if case["way"] != "backward":
        # a padded place keeps the state
        keep = torch.where(live, f * go, 1.0).transpose(0, 1).contiguous()
        add = (i * v * live).transpose(0, 1).contiguous()
        out = torch.empty_like(add)
        for t in range(length):
            state = torch.addcmul(add[t], keep[t], state, out=out[t])
        return {"h": out.transpose(0, 1) * live, "h_last": state}
    h = s["h"].double().masked_fill(~live, 0)
    keep = torch.where(live, f * go, 1.0).transpose(0, 1).contiguous()
    dh = s["dh"].double().masked_fill(~live, 0).transpose(0, 1).contiguous()
    delta = torch.empty_like(dh)
    grad = s["dh_last"].double()  # gradient of the state after token t
    for t in range(length - 1, -1, -1):
        torch.add(dh[t], grad, out=delta[t])
        grad = keep[t] * delta[t]
    delta = delta.transpose(0, 1) * live
    prev = torch.cat([state[:, None], h[:, :-1]], 1) * go
    return {"dg": delta * (prev - v) * f * i, "dv": i * delta, "dh0": grad}

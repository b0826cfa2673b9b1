"""Cases of the attention operators around the fast-weight layer: norms of queries and keys for each head
with the position rotation (forward, backward, and the serving form that appends to a paged cache), attention
over packed prompts (forward, and training steps with the backward), and attention of one new token over a
paged key-value cache.

`run` computes a case in plain torch operations where `own` is false and through
chunked_weight_mlp_amd.attention where it is true. Head layouts are those of the repository's layer widths
(d 2560 and d 2048) and odd ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # --- norms of queries and keys, rotation ---
        # decoding: one token of each of 32 sequences, keys and values appended to the paged cache
        dict(name="heads_token", op="heads", way="append", dtype="bf16", n=32, hq=32, hk=8, dh=128, rotary=128,
             interleaved=False, page=64, pages=8, cut=1),
        # prefill of a 32k document, queries and keys out of one fused projection
        dict(name="heads_prompt", op="heads", way="forward", dtype="bf16", n=32768, hq=32, hk=8, dh=128,
             rotary=128, interleaved=False),
        # training on 8 x 16k tokens
        dict(name="heads_train", op="heads", way="backward", dtype="bf16", n=131072, hq=16, hk=8, dh=128,
             rotary=128, interleaved=False),
        # a small fp32 model: odd row count, a third of each head rotated, neighbouring pairs
        dict(name="heads_odd_f32", op="heads", way="backward", dtype="f32", n=1021, hq=6, hk=3, dh=72, rotary=24,
             interleaved=True),
        # --- attention over prompts ---
        # prefill of one 32k document
        dict(name="prompt_32k", op="prompt", way="forward", dtype="bf16", n=32768, seqs=1, prefix=0, hq=32, hk=8,
             dh=128, window=0, cut=1),
        # prefill of a batch of 24 prompts of different lengths, packed
        dict(name="prompt_packed", op="prompt", way="forward", dtype="bf16", n=16411, seqs=24, prefix=0, hq=32,
             hk=8, dh=128, window=0, cut=2),
        # the next 2048 tokens of two documents, sliding window, over the 8192 keys before them
        dict(name="prompt_window", op="prompt", way="forward", dtype="bf16", n=4096, seqs=2, prefix=8192, hq=32,
             hk=8, dh=128, window=4096, cut=0),
        # a training step's packed documents, forward and backward
        dict(name="prompt_train", op="prompt", way="train", dtype="bf16", n=16384, seqs=6, prefix=0, hq=16, hk=8,
             dh=128, window=0, cut=3),
        # a small fp32 model trained on short documents, odd sizes
        dict(name="prompt_odd_f32", op="prompt", way="train", dtype="f32", n=701, seqs=5, prefix=0, hq=6, hk=2,
             dh=40, window=0, cut=4),
        # --- one new token over the cache ---
        # decoding one sequence behind a 128k document
        dict(name="step_128k", op="step", dtype="bf16", n=131072, seqs=1, hq=32, hk=8, dh=128, window=0, page=64,
             cut=0),
        # decoding 64 sequences of different lengths
        dict(name="step_batch", op="step", dtype="bf16", n=131072, seqs=64, hq=32, hk=8, dh=128, window=0, page=16,
             cut=5),
        # a few short fp32 sequences, pages and heads of odd sizes: latency
        dict(name="step_short_f32", op="step", dtype="f32", n=301, seqs=4, hq=6, hk=3, dh=72, window=0, page=24,
             cut=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _layout(rng):
    """Heads of queries and keys, and their width."""
    dh = rng.choice([128, 128, 128, 64, 64, 96, 80, 72, 40, 33])
    hk = rng.choice([1, 2, 3, 4, 8, 8])
    return hk * rng.choice([1, 2, 4, 4, 5, 8]), hk, dh


def draw(rng):
    op = rng.choice(["heads", "prompt", "prompt", "step", "step"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    hq, hk, dh = _layout(rng)
    cut = rng.randrange(1 << 20)
    if op == "heads":
        way = rng.choice(["forward", "append", "backward"])
        rotary = rng.choice([dh // 2 * 2, dh // 2 * 2, dh // 4 * 2])
        case = dict(op=op, way=way, dtype=dtype, n=_log(rng, 1, 512 if way == "append" else 32768), hq=hq, hk=hk,
                    dh=dh, rotary=rotary, interleaved=rng.random() < 0.3)
        if way == "append":
            case.update(page=rng.choice([16, 64, 24]), pages=rng.choice([1, 3, 8]), cut=cut)
        return case
    if op == "prompt":
        way = rng.choice(["forward", "train"])
        window = 0 if rng.random() < 0.7 else _log(rng, 1, 4096)
        seqs = _log(rng, 1, 64)
        # pairs of tokens bound the work; few sequences pair nearly all of them
        most = int((2 ** 30 / (hq * (3 if way == "train" else 1) * (2 if dtype == "f32" else 1))
                    * 128 / max(dh, 64) * min(seqs, 8)) ** 0.5)
        n = _log(rng, seqs, max(seqs, most))
        return dict(op=op, way=way, dtype=dtype, n=n, seqs=seqs,
                    prefix=0 if rng.random() < 0.7 else _log(rng, 1, max(1, most // seqs // 2)), hq=hq, hk=hk, dh=dh,
                    window=window, cut=cut)
    seqs = _log(rng, 1, 128)
    most = 131072 * 8 * 128 // (hk * dh * (2 if dtype == "f32" else 1))
    return dict(op=op, dtype=dtype, n=_log(rng, seqs, max(seqs, min(262144, most))), seqs=seqs, hq=hq, hk=hk, dh=dh,
                window=0 if rng.random() < 0.8 else _log(rng, 1, 4096), page=rng.choice([16, 64, 64, 128, 24, 1]),
                cut=cut)


def _lens(case):
    """The sequences' lengths: n tokens cut at random places (in equal parts where cut is 0)."""
    n, k = case["n"], case["seqs"]
    if case["cut"] == 0:
        return [n // k + (i < n % k) for i in range(k)]
    rng = random.Random(case["cut"])
    cuts = sorted(rng.randint(0, n) for _ in range(k - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [n])]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _offsets(lens):
    at = [0]
    for m in lens:
        at.append(at[-1] + m)
    return at


def prepare(case, seed):
    g, t = _gen(seed), TYPES[case["dtype"]]
    n, hq, hk, dh = (case[k] for k in ("n", "hq", "hk", "dh"))
    s = dict(case=case)
    if case["op"] == "heads":
        qkv = _normal(g, (n, (hq + 2 * hk) * dh), t)
        s["q"], s["k"], s["v"] = (x.view(n, -1, dh) for x in qkv.split([hq * dh, hk * dh, hk * dh], 1))
        s["q_gamma"], s["k_gamma"] = ((1 + _normal(g, (dh,), torch.float32, 0.2)).to(t) for _ in range(2))
        r = case["rotary"]
        s["inv_freq"] = 1e6 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / max(r, 1))
        if case["way"] == "append":
            # every sequence's next place, in pages in any order of a pool with some to spare
            page, pages = case["page"], case["pages"]
            s["pos"] = torch.randint(0, page * pages, (n,), generator=g, device=DEV, dtype=torch.int32)
            order = torch.randperm(n * pages + 3, generator=g, device=DEV).to(torch.int32)
            s["table"] = order[:n * pages].view(n, pages).contiguous()
            s["k_pages"], s["v_pages"] = (_normal(g, (n * pages + 3, hk, page, dh), t) for _ in range(2))
        else:
            first = int(torch.randint(0, 131072, (1,), generator=g, device=DEV))
            s["pos"] = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
        if case["way"] == "backward":
            s["dq"], s["dk"] = _normal(g, (n, hq, dh), t), _normal(g, (n, hk, dh), t)
        if own:
            from chunked_weight_mlp_amd import attention
            s["op"] = attention.HeadNorm(s["q_gamma"], s["k_gamma"], s["inv_freq"], eps=EPS,
                                         interleaved=case["interleaved"])
            if case["way"] == "append":
                s["cache"] = attention.KVCache(s["k_pages"], s["v_pages"])
        return s
    lens = s["lens"] = _lens(case)
    if case["op"] == "prompt":
        k_lens = s["k_lens"] = [m + case["prefix"] for m in lens]
        s["offsets"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=DEV)
        s["k_offsets"] = torch.tensor(_offsets(k_lens), dtype=torch.int32, device=DEV)
        # normed heads: scores of standard deviation 2
        s["q"] = _normal(g, (n, hq, dh), t, 2.0)
        s["k"], s["v"] = _normal(g, (sum(k_lens), hk, dh), t), _normal(g, (sum(k_lens), hk, dh), t)
        if case["way"] == "train":
            s["do"] = _normal(g, (n, hq, dh), t)
        return s
    page = case["page"]
    pages = [-(-m // page) for m in lens]
    order = torch.randperm(sum(pages) + 3, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), max(max(pages), 1)), -1, dtype=torch.int32)
    for i, (at, m) in enumerate(zip(_offsets(pages), pages)):
        table[i, :m] = order[at:at + m]
    s["table"], s["len"] = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["k_pages"], s["v_pages"] = (_normal(g, (sum(pages) + 3, hk, page, dh), t) for _ in range(2))
    s["q"] = _normal(g, (len(lens), hq, dh), t, 2.0)
    if own:
        from chunked_weight_mlp_amd import attention
        s["cache"] = attention.KVCache(s["k_pages"], s["v_pages"])
    return s


# ---- plain forms -----------------------------------------------------------------------------


def _turn(x, cos, sin, interleaved, back=False):
    """The rotation of the first 2 cos.shape[-1] channels of [n, heads, dh], or its transpose."""
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if back:
        sin = -sin
    head, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _plain_heads(s):
    case = s["case"]
    t, way = s["q"].dtype, case["way"]
    # angles of far positions need 64 bits
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for name in ("q", "k"):
        x, gamma = s[name].float(), s[name + "_gamma"].float()
        xh = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if way != "backward":
            out[name] = _turn(xh * gamma, cos, sin, case["interleaved"]).to(t)
            continue
        g = _turn(s["d" + name].float(), cos, sin, case["interleaved"], back=True)
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        w = g * gamma
        out["d" + name] = ((w - xh * (w * xh).mean(-1, keepdim=True)) * rstd).to(t)
        out["d" + name + "_gamma"] = (g * xh).sum((0, 1))
    if way == "append":
        pos = s["pos"].long()
        row = torch.gather(s["table"].long(), 1, (pos // case["page"])[:, None])[:, 0]
        s["k_pages"][row, :, pos % case["page"]] = out.pop("k")
        s["v_pages"][row, :, pos % case["page"]] = s["v"]
        out["k_pages"], out["v_pages"] = s["k_pages"], s["v_pages"]
    return out


def _plain_prompt(s):
    """One sequence after another; rows in blocks where a score matrix would be too large."""
    case = s["case"]
    hq, hk, dh, window = (case[k] for k in ("hq", "hk", "dh", "window"))
    group, scale, t = hq // hk, dh ** -0.5, s["q"].dtype
    train = case["way"] == "train"
    o, lse = torch.empty_like(s["q"]), torch.empty((hq, case["n"]), dtype=torch.float32, device=DEV)
    dq, dk, dv = (torch.empty_like(s[x]) for x in "qkv") if train else (None, None, None)
    at = k_at = 0
    for lq, lk in zip(s["lens"], s["k_lens"]):
        k, v = (s[x][k_at:k_at + lk].float().transpose(0, 1) for x in "kv")
        if train:
            sum_k, sum_v = torch.zeros_like(k), torch.zeros_like(v)
        rows = max(1, (1 << 30) // max(1, hq * lk))
        for r0 in range(0, lq, rows):
            r1 = min(r0 + rows, lq)
            end = r1 + lk - lq                                    # keys that some row sees
            i = torch.arange(r0, r1, device=DEV)[:, None] + (lk - lq)
            j = torch.arange(end, device=DEV)
            hidden = j > i
            if window:
                hidden = hidden | (j <= i - window)
            q = s["q"][at + r0:at + r1].float().transpose(0, 1).reshape(hk, group * (r1 - r0), dh)
            sc = ((q @ k[:, :end].transpose(1, 2)) * scale).view(hk, group, r1 - r0, end)
            sc = sc.masked_fill_(hidden, float("-inf"))
            m = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - m)
            l = p.sum(-1, keepdim=True)
            p = (p / l).view(hk, -1, end)
            lse[:, at + r0:at + r1] = (m + l.log()).view(hq, -1)
            o[at + r0:at + r1] = (p @ v[:, :end]).view(hq, -1, dh).transpose(0, 1).to(t)
            if train:
                do = s["do"][at + r0:at + r1].float().transpose(0, 1).reshape(hk, -1, dh)
                dp = do @ v[:, :end].transpose(1, 2)
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                dq[at + r0:at + r1] = (ds @ k[:, :end]).view(hq, -1, dh).transpose(0, 1).to(t)
                sum_k[:, :end] += ds.transpose(1, 2) @ q
                sum_v[:, :end] += p.transpose(1, 2) @ do
        if train:
            dk[k_at:k_at + lk] = sum_k.transpose(0, 1).to(t)
            dv[k_at:k_at + lk] = sum_v.transpose(0, 1).to(t)
        at, k_at = at + lq, k_at + lk
    out = {"o": o, "lse": lse}
    return {**out, "dq": dq, "dk": dk, "dv": dv} if train else out


def _plain_step(s):
    """The sequences' pages gathered to the longest one's length."""
    case = s["case"]
    hq, hk, dh = (case[k] for k in ("hq", "hk", "dh"))
    b = len(s["lens"])
    at = s["table"].long().clamp_min(0)
    k, v = (s[x][at].float().transpose(1, 2).reshape(b, hk, -1, dh) for x in ("k_pages", "v_pages"))
    j = torch.arange(k.shape[2], device=DEV)
    hidden = j >= s["len"][:, None]
    if case["window"]:
        hidden = hidden | (j < s["len"][:, None] - case["window"])
    q = s["q"].float().view(b, hk, hq // hk, dh)
    sc = (q @ k.transpose(2, 3) * dh ** -0.5).masked_fill_(hidden[:, None, None], float("-inf"))
    # a sequence of no tokens has no key: zeros
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    o = (p @ v.masked_fill_(hidden[:, None, :, None], 0.0)) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return {"o": o.view(b, hq, dh).to(s["q"].dtype)}


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"heads": _plain_heads, "prompt": _plain_prompt, "step": _plain_step}[case["op"]](s)
    from chunked_weight_mlp_amd import attention
    if case["op"] == "heads":
        if case["way"] == "forward":
            q, k = s["op"].forward(s["q"], s["k"], s["pos"])
            return {"q": q, "k": k}
        if case["way"] == "append":
            q = s["op"].append(s["q"], s["k"], s["v"], s["pos"], s["cache"], s["table"])
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return s["op"].backward(s["q"], s["k"], s["pos"], s["dq"], s["dk"])
    if case["op"] == "step":
        return {"o": attention.attention_step(s["q"], s["cache"], s["table"], s["len"], window=case["window"])}
    at = dict(offsets=s["offsets"], k_offsets=s["k_offsets"], window=case["window"])
    o, lse = attention.attention_forward(s["q"], s["k"], s["v"], **at)
    out = {"o": o, "lse": lse}
    if case["way"] == "train":
        out.update(attention.attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], **at))
    return out


def _pairs(lq, lk, window):
    """Pairs of a query and a key that it sees, of one sequence whose last query sees the last key."""
    full = lq * (lk - lq) + lq * (lq + 1) // 2
    if not window or window >= lk:
        return full
    # the m-th key from the end of row i's is out of the window from m = window on
    m = lk - window                     # rows that see more than a window, by what they see too much
    less = lq * (lq + 1) // 2 + lq * (lk - lq - window) if lk - lq >= window else m * (m + 1) // 2
    return full - less


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hk, dh = (case[k] for k in ("hq", "hk", "dh"))
    if case["op"] == "heads":
        el = case["n"] * (hq + hk) * dh
        passes = 3 if case["way"] == "backward" else 2
        v = 2 * case["n"] * hk * dh if case["way"] == "append" else 0
        return {"bytes": (passes * el + v) * e + 4 * case["n"], "flops": (20 if passes == 3 else 10) * el}
    lens, window = _lens(case), case["window"]
    if case["op"] == "step":
        live = sum(min(m, window) if window else m for m in lens)
        return {"bytes": (2 * live * hk + 2 * len(lens) * hq) * dh * e, "flops": 4 * live * hq * dh}
    n, n_k = case["n"], case["n"] + case["seqs"] * case["prefix"]
    pairs = sum(_pairs(m, m + case["prefix"], window) for m in lens)
    if case["way"] == "train":
        # q, k, v, do -> o, lse, dq, dk, dv
        return {"bytes": (4 * n * hq + 4 * n_k * hk) * dh * e + 4 * n * hq, "flops": 14 * pairs * hq * dh}
    return {"bytes": (2 * n * hq + 2 * n_k * hk) * dh * e + 4 * n * hq, "flops": 4 * pairs * hq * dh}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _rotations(s, case):
    """[n, dh, dh] would be large: the rotation as a complex factor of each pair."""
    turns = s["pos"].double().view(-1, 1, 1) * s["inv_freq"].view(1, 1, -1)
    return torch.polar(torch.ones_like(turns), turns)


def _pairs_of(x, case):
    """[n, heads, dh] as complex pairs of the rotated channels, and the rest."""
    r = case["rotary"]
    head = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
    if not case["interleaved"]:
        head = head.transpose(-1, -2)
    return torch.view_as_complex(head.contiguous()), x[..., r:]


def _from_pairs(z, rest, case):
    head = torch.view_as_real(z)
    if not case["interleaved"]:
        head = head.transpose(-1, -2)
    return torch.cat([head.flatten(-2), rest], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        factor, out, dh = _rotations(s, case), {}, case["dh"]
        for name in ("q", "k"):
            x, gamma = s[name].double(), s[name + "_gamma"].double()
            norm = ((x * x).sum(-1, keepdim=True) / dh + EPS).sqrt()
            if case["way"] != "backward":
                z, rest = _pairs_of(x / norm * gamma, case)
                out[name] = _from_pairs(z * factor, rest, case)
                continue
            z, rest = _pairs_of(s["d" + name].double(), case)
            g = _from_pairs(z * factor.conj(), rest, case)
            # y = x gamma / norm(x): d norm / d x_c = x_c / (dh norm)
            inner = (g * gamma * x).sum(-1, keepdim=True)
            out["d" + name] = g * gamma / norm - x * inner / (dh * norm ** 3)
            out["d" + name + "_gamma"] = torch.einsum("nhc,nhc->c", g, x / norm)
        if case["way"] == "append":
            pages = {x: s[x].double() for x in ("k_pages", "v_pages")}
            for i, p in enumerate(s["pos"].tolist()):
                at, slot = int(s["table"][i, p // case["page"]]), p % case["page"]
                pages["k_pages"][at, :, slot] = out["k"][i]
                pages["v_pages"][at, :, slot] = s["v"][i].double()
            out = {"q": out["q"], **pages}
        return out
    hq, hk, dh, window = (case[k] for k in ("hq", "hk", "dh", "window"))
    group = hq // hk
    if case["op"] == "step":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for i, m in enumerate(s["lens"]):
            if m == 0:
                continue
            at = s["table"][i, :-(-m // case["page"])].long()
            lo = max(0, m - window) if window else 0
            for h in range(hk):
                k, v = (s[x][at, h].reshape(-1, dh)[lo:m].double() for x in ("k_pages", "v_pages"))
                p = torch.softmax(s["q"][i, h * group:(h + 1) * group].double() @ k.t() / math.sqrt(dh), -1)
                o[i, h * group:(h + 1) * group] = p @ v
        return {"o": o}
    n, train = case["n"], case["way"] == "train"
    out = {"o": torch.empty((n, hq, dh), dtype=torch.float64, device=DEV),
           "lse": torch.empty((hq, n), dtype=torch.float64, device=DEV)}
    if train:
        out["dq"] = torch.empty_like(out["o"])
        out["dk"], out["dv"] = (torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
    at = k_at = 0
    for lq, lk in zip(s["lens"], s["k_lens"]):
        ks = slice(k_at, k_at + lk)
        step = max(1, (1 << 28) // max(1, lk))
        for h in range(hq):
            k, v = s["k"][ks, h // group].double(), s["v"][ks, h // group].double()
            for r in range(0, lq, step):
                rows = slice(at + r, at + min(r + step, lq))
                q = s["q"][rows, h].double()
                last = torch.arange(rows.start, rows.stop, device=DEV).sub_(at - (lk - lq))  # last key seen
                back = last[:, None] - torch.arange(lk, device=DEV)
                seen = back >= 0
                if window:
                    seen &= back < window
                a = torch.where(seen, q.mm(k.t()) / math.sqrt(dh), -math.inf)
                out["lse"][h, rows] = torch.logsumexp(a, 1)
                p = torch.exp(a - out["lse"][h, rows][:, None])
                out["o"][rows, h] = p.mm(v)
                if train:
                    do = s["do"][rows, h].double()
                    out["dv"][ks, h // group] += p.t().mm(do)
                    delta = (do * out["o"][rows, h]).sum(1, keepdim=True)
                    da = p * (do.mm(v.t()) - delta) / math.sqrt(dh)
                    out["dq"][rows, h] = da.mm(k)
                    out["dk"][ks, h // group] += da.t().mm(q)
        at, k_at = at + lq, k_at + lk
    return out

"""The attention operators beside the fast-weight layer (include/ipttt_attention.h) over
libipttt's HIP kernels: norms of queries and keys for each head with the rotation by
position, attention over packed prompts, and attention of one new token over a paged
cache; the first two with their backward.

The `ipttt_*` functions are the C entry points with tensors for pointers. HeadNorm holds
the norms' weights, KVCache a paged cache; attention_forward / _backward / _step allocate
their outputs and workspace. Tensors, streams, errors and gradients are as in `block`:
tensors on the current device, the current stream or `stream=`, ipttt.IptttError for what
is refused, outputs detached.

Tensors of heads are [tokens, heads, head_dim], float32 or bfloat16, with contiguous
channels; tokens and heads may lie in any order and apart (slices of a fused projection).
"""
from __future__ import annotations

import ctypes

import torch

from . import ipttt as _b
from .block import (_DENSE, _call_on, _check, _dense, _dtype_of, _invalid, _is, _on, _p, _ref, _stream,
                    _temp)

EXPORTS = (
    "ipttt_headnorm_forward", "ipttt_headnorm_append", "ipttt_headnorm_backward_workspace_bytes",
    "ipttt_headnorm_backward", "ipttt_attention_forward_workspace_bytes", "ipttt_attention_forward",
    "ipttt_attention_backward_workspace_bytes", "ipttt_attention_backward", "ipttt_attention_step_workspace_bytes", "ipttt_attention_step",
)


class Heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int)]


class PageTable(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("width", ctypes.c_int32)]


class HeadNormDesc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("n_q", ctypes.c_int64),
                ("n_k", ctypes.c_int64), ("q_offsets", ctypes.c_void_p), ("k_offsets", ctypes.c_void_p)]


class StepDesc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def load() -> ctypes.CDLL:
    """The library with this header's signatures; raises if it is not built."""
    global _lib
    if _lib is None:
        lib = _b.load()
        vp, i64, sz, P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER
        h = P(Heads)
        sig = {
            "ipttt_headnorm_forward": [P(HeadNormDesc), h, h, vp, i64, h, h, vp],
            "ipttt_headnorm_append": [P(HeadNormDesc), h, h, h, vp, vp, i64, h, P(KVCacheDesc), P(PageTable),
                                      vp],
            "ipttt_headnorm_backward": [P(HeadNormDesc), h, h, vp, h, h, i64, h, h, vp, vp, vp, sz, vp],
            "ipttt_attention_forward": [P(AttentionDesc), h, h, h, h, vp, vp, sz, vp],
            "ipttt_attention_backward": [P(AttentionDesc), h, h, h, h, vp, h, h, h, h, vp, sz, vp],
            "ipttt_attention_step": [P(StepDesc), h, P(KVCacheDesc), P(PageTable), vp, h, vp, vp, sz, vp],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        for name, args in {
                "ipttt_headnorm_backward_workspace_bytes": [P(HeadNormDesc), i64],
                "ipttt_attention_forward_workspace_bytes": [P(AttentionDesc)],
                "ipttt_attention_backward_workspace_bytes": [P(AttentionDesc)],
                "ipttt_attention_step_workspace_bytes": [P(StepDesc), P(KVCacheDesc), P(PageTable)]}.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, sz
        _lib = lib
    return _lib


# ---- the C entry points -----------------------------------------------------------------


def ipttt_headnorm_forward(desc, q, k, pos, n, q_out, k_out, stream=None) -> None:
    _check(load().ipttt_headnorm_forward(_ref(desc), _ref(q), _ref(k), _p(pos), n, _ref(q_out), _ref(k_out),
                                         _stream(stream)))


def ipttt_headnorm_append(desc, q, k, v, pos, seqs, n, q_out, cache, table, stream=None) -> None:
    _check(load().ipttt_headnorm_append(_ref(desc), _ref(q), _ref(k), _ref(v), _p(pos), _p(seqs), n, _ref(q_out),
                                        _ref(cache), _ref(table), _stream(stream)))


def ipttt_headnorm_backward_workspace_bytes(desc, n: int) -> int:
    return load().ipttt_headnorm_backward_workspace_bytes(_ref(desc), n)


def ipttt_headnorm_backward(desc, q, k, pos, dq, dk, n, dx_q, dx_k, dq_gamma, dk_gamma, workspace,
                            workspace_bytes, stream=None) -> None:
    _check(load().ipttt_headnorm_backward(_ref(desc), _ref(q), _ref(k), _p(pos), _ref(dq), _ref(dk), n,
                                          _ref(dx_q), _ref(dx_k), _p(dq_gamma), _p(dk_gamma), _p(workspace),
                                          workspace_bytes, _stream(stream)))


def ipttt_attention_forward_workspace_bytes(desc) -> int:
    return load().ipttt_attention_forward_workspace_bytes(_ref(desc))


def ipttt_attention_forward(desc, q, k, v, o, lse, workspace, workspace_bytes, stream=None) -> None:
    _check(load().ipttt_attention_forward(_ref(desc), _ref(q), _ref(k), _ref(v), _ref(o), _p(lse), _p(workspace),
                                          workspace_bytes, _stream(stream)))


def ipttt_attention_backward_workspace_bytes(desc) -> int:
    return load().ipttt_attention_backward_workspace_bytes(_ref(desc))


def ipttt_attention_backward(desc, q, k, v, o, lse, dy, dq, dk, dv, workspace, workspace_bytes,
                             stream=None) -> None:
    _check(load().ipttt_attention_backward(_ref(desc), _ref(q), _ref(k), _ref(v), _ref(o), _p(lse), _ref(dy),
                                           _ref(dq), _ref(dk), _ref(dv), _p(workspace), workspace_bytes,
                                           _stream(stream)))


def ipttt_attention_step_workspace_bytes(desc, cache, table) -> int:
    return load().ipttt_attention_step_workspace_bytes(_ref(desc), _ref(cache), _ref(table))


def ipttt_attention_step(desc, q, cache, table, lens, o, lse, workspace, workspace_bytes, stream=None) -> None:
    _check(load().ipttt_attention_step(_ref(desc), _ref(q), _ref(cache), _ref(table), _p(lens), _ref(o), _p(lse),
                                       _p(workspace), workspace_bytes, _stream(stream)))


# ---- operators over tensors ---------------------------------------------------------------


def _heads(name, t, shape, dtype, device):
    """A tensor [tokens, heads, head_dim] as the library takes it."""
    if t.shape != shape:
        raise _invalid(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        _is(name, t, dtype, device)
    tok, head, ch = t.stride()
    if ch != 1 and shape[2] > 1 and t.numel():
        raise _invalid(f"{name} must have its channels contiguous")
    return Heads(t.data_ptr(), tok, head)


def _int32(name, v):
    """v as a field of 32 bits, which ctypes would cut it to."""
    if not -2 ** 31 <= v < 2 ** 31:
        raise _invalid(f"{name}={v} does not fit 32 bits")
    return v


def _three(name, t):
    if t.dim() != 3 or 0 in t.shape[1:]:
        raise _invalid(f"{name} must be [tokens, heads, head_dim], the last two > 0")
    n, heads, dh = t.shape
    if heads >= 2 ** 31 or dh >= 2 ** 31:
        raise _invalid(f"{name} has shape {(n, heads, dh)}: heads or head_dim do not fit 32 bits")
    return t.shape


class KVCache:
    """A paged cache of keys and values: k, v [pages, k_heads, page_size, head_dim]. Which pages
    hold a sequence is said by a table in each call, int32 [sequences, pages each may have]:
    token t of sequence s is in page table[s, t // page_size] at t % page_size. Numbers
    outside the cache (-1) are no page."""

    def __init__(self, k, v):
        if k.dim() != 4 or 0 in k.shape[1:]:
            raise _invalid("k must be [pages, k_heads, page_size, head_dim], all but the pages > 0")
        dt = _dtype_of(k)
        for name, size in zip(("pages", "k_heads", "page_size", "head_dim"), k.shape):
            _int32(name, size)
        self.k = _dense("k", k, k.shape, k.dtype, k.device)
        self.v = _dense("v", v, k.shape, k.dtype, k.device)
        self.pages, self.k_heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), self.pages, self.page_size, self.k_heads, self.head_dim,
                                dt)
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, pages, k_heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of pages that nothing has been written to."""
        return cls(*(torch.empty((pages, k_heads, page_size, head_dim), dtype=dtype, device=device)
                     for _ in range(2)))

    def table(self, table):
        """The call's form of a page table."""
        if table.dim() != 2:
            raise _invalid("table must be [sequences, pages]")
        if max(table.shape) >= 2 ** 31:
            raise _invalid(f"table has shape {tuple(table.shape)}, which does not fit 32 bits")
        _is("table", table, torch.int32, self.device)
        if table.numel() and table.shape[1] > 1 and table.stride(1) != 1:
            raise _invalid("table must have its rows contiguous")
        return PageTable(table.data_ptr(), table.stride(0), table.shape[0], table.shape[1])


class HeadNorm:
    """Norms of queries and keys for each head (root mean square, weights q_gamma, k_gamma
    [head_dim] or None for a tensor that is not normed) and the rotation of the first
    2 * len(inv_freq) channels by pos * inv_freq (radians a position, kept in 64 bits):
    pairs are channels i and i + len(inv_freq), or 2 i and 2 i + 1 if interleaved.
    Without gammas, say dtype and head_dim. All tensors are on inv_freq's device."""

    def __init__(self, q_gamma, k_gamma, inv_freq, eps: float = 1e-6, interleaved: bool = False, head_dim=None,
                 dtype=None):
        like = q_gamma if q_gamma is not None else k_gamma
        if like is not None:
            if like.dim() != 1 or like.numel() == 0:
                raise _invalid("gammas must be [head_dim], head_dim > 0")
            head_dim, dtype = like.shape[0], like.dtype
        elif head_dim is None or dtype is None:
            raise _invalid("without gammas, head_dim and dtype must be given")
        if inv_freq.dim() != 1 or not inv_freq.is_floating_point():
            raise _invalid("inv_freq must be a vector of floating numbers")
        _int32("head_dim", head_dim), _int32("rotary", 2 * inv_freq.numel())
        self.head_dim, self.dtype, self.device = head_dim, dtype, inv_freq.device
        dt = _b._DT.get(dtype)
        if dt is None:
            _dtype_of(torch.empty(0, dtype=dtype))
        self.q_gamma, self.k_gamma = (
            None if g is None else _dense(name, g, (head_dim,), dtype, self.device)
            for name, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)))
        self.inv_freq = inv_freq.detach().to(torch.float64).contiguous()
        self.eps, self.interleaved, self._dt = eps, bool(interleaved), dt
        self._descs = {}

    def _desc(self, hq, hk):
        """The descriptor for these numbers of heads."""
        d = self._descs.get((hq, hk))
        if d is None:
            d = self._descs[hq, hk] = ctypes.byref(HeadNormDesc(
                hq, hk, self.head_dim, 2 * self.inv_freq.numel(), self.interleaved, self._dt, self.eps,
                _p(self.q_gamma), _p(self.k_gamma), self.inv_freq.data_ptr()))
        return d

    def _held(self):
        return self.q_gamma, self.k_gamma, self.inv_freq

    def _checked(self, q, k, pos):
        """(q, k as heads, their numbers, tokens, the descriptor)."""
        n, hq, dh = _three("q", q)
        hk = _three("k", k)[1]
        dtype, dev = self.dtype, self.device
        qh = _heads("q", q, (n, hq, self.head_dim), dtype, dev)
        kh = _heads("k", k, (n, hk, self.head_dim), dtype, dev)
        _dense("pos", pos, (n,), torch.int32, dev)
        return qh, kh, hq, hk, n, self._desc(hq, hk)

    def forward(self, q, k, pos, stream=None):
        """Returns (q, k) normed and rotated, dense. q, k: [tokens, heads, head_dim]; pos: int32
        [tokens]."""
        if stream is not None:
            return _call_on(stream, self.forward, (q, k, pos), self._held())
        qh, kh, _, _, n, desc = self._checked(q, k, pos)
        st = _on(self.device)
        qo, ko = (torch.empty_like(t, memory_format=_DENSE) for t in (q, k))
        _check(load().ipttt_headnorm_forward(
            desc, qh, kh, pos.data_ptr(), n, _heads("q_out", qo, q.shape, self.dtype, self.device),
            _heads("k_out", ko, k.shape, self.dtype, self.device), st))
        return qo, ko

    def append(self, q, k, v, pos, cache, table, seqs=None, stream=None):
        """As forward, with the keys' results and v written to the cache instead: token t at
        position pos[t] of sequence seqs[t] (int32 [tokens]; None: of sequence t). Returns q.
        A token whose place the table does not hold (a negative position marks padding) is
        not written. No two tokens may have the same place."""
        if stream is not None:
            return _call_on(stream, self.append, (q, k, v, pos, cache, table, seqs),
                            (*self._held(), cache.k, cache.v))
        qh, kh, _, hk, n, desc = self._checked(q, k, pos)
        dtype, dev = self.dtype, self.device
        vh = _heads("v", v, k.shape, dtype, dev)
        if seqs is not None:
            _dense("seqs", seqs, (n,), torch.int32, dev)
        if cache.device != dev:
            raise _invalid(f"the cache is on {cache.device}, expected {dev}")
        tab = cache.table(table)
        st = _on(dev)
        qo = torch.empty_like(q, memory_format=_DENSE)
        _check(load().ipttt_headnorm_append(desc, qh, kh, vh, pos.data_ptr(), _p(seqs), n,
                                            _heads("q_out", qo, q.shape, dtype, dev), cache._ref, tab, st))
        return qo

    def backward(self, q, k, pos, dq, dk, stream=None):
        """Gradients of forward from its inputs and dL/dq, dL/dk of its results: {"dq", "dk"}
        dense, in the activations' dtype, and fp32 {"dq_gamma", "dk_gamma"} (None for a
        tensor that is not normed)."""
        if stream is not None:
            return _call_on(stream, self.backward, (q, k, pos, dq, dk), self._held())
        qh, kh, hq, hk, n, desc = self._checked(q, k, pos)
        dtype, dev = self.dtype, self.device
        gq, gk = _heads("dq", dq, q.shape, dtype, dev), _heads("dk", dk, k.shape, dtype, dev)
        st = _on(dev)
        oq, ok = (torch.empty_like(t, memory_format=_DENSE) for t in (q, k))
        dg = [None if g is None else torch.empty(self.head_dim, dtype=torch.float32, device=dev)
              for g in (self.q_gamma, self.k_gamma)]
        need = load().ipttt_headnorm_backward_workspace_bytes(desc, n)
        ws = _temp(need, dev)
        _check(load().ipttt_headnorm_backward(
            desc, qh, kh, pos.data_ptr(), gq, gk, n, _heads("dx_q", oq, q.shape, dtype, dev),
            _heads("dx_k", ok, k.shape, dtype, dev), _p(dg[0]), _p(dg[1]), ws.data_ptr(), need, st))
        return {"dq": oq, "dk": ok, "dq_gamma": dg[0], "dk_gamma": dg[1]}


def _attention(q, k, v, offsets, k_offsets, causal, window, scale):
    """The descriptor of an attention over prompts, and its inputs as heads."""
    n, hq, dh = _three("q", q)
    nk, hk, _ = _three("k", k)
    dtype, dev = q.dtype, q.device
    dt = _dtype_of(q)
    views = [_heads(name, t, (m, heads, dh), dtype, dev)
             for name, t, m, heads in (("q", q, n, hq), ("k", k, nk, hk), ("v", v, nk, hk))]
    if k_offsets is None:
        if nk != n and offsets is not None:
            raise _invalid(f"k has {nk} rows for {n} queries: their sequences need k_offsets")
        k_offsets = offsets
    if (offsets is None) != (k_offsets is None):
        raise _invalid("k_offsets without offsets")
    batch = 1
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() == 0:
            raise _invalid("offsets must be [sequences + 1]")
        _int32("sequences", offsets.numel() - 1)
        _dense("offsets", offsets, offsets.shape, torch.int32, dev)
        _dense("k_offsets", k_offsets, offsets.shape, torch.int32, dev)
        batch = offsets.numel() - 1
    scale = dh ** -0.5 if scale is None else scale
    return AttentionDesc(hq, hk, dh, batch, bool(causal), _int32("window", window), dt, scale, n, nk, _p(offsets),
                         _p(k_offsets)), views


def attention_forward(q, k, v, offsets=None, k_offsets=None, causal: bool = True, window: int = 0, scale=None,
                      stream=None):
    """softmax(scale q k^T) v of packed sequences: q [tokens, q_heads, head_dim], k, v
    [keys, k_heads, head_dim], q_heads a multiple of k_heads. offsets: int32
    [sequences + 1], where each sequence's queries begin (None: one sequence); k_offsets:
    the same of its keys (None: as the queries). Causal attention lets the last query see
    the last key; window > 0 leaves each query its last `window` keys. scale: None for
    head_dim ** -0.5. Returns (o, lse): o like q, dense, and fp32 [q_heads, tokens]."""
    if stream is not None:
        return _call_on(stream, attention_forward, (q, k, v, offsets, k_offsets, causal, window, scale))
    desc, views = _attention(q, k, v, offsets, k_offsets, causal, window, scale)
    st = _on(q.device)
    o = torch.empty_like(q, memory_format=_DENSE)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    ref = ctypes.byref(desc)
    need = load().ipttt_attention_forward_workspace_bytes(ref)
    ws = _temp(need, q.device)
    _check(load().ipttt_attention_forward(ref, *views, _heads("o", o, q.shape, q.dtype, q.device),
                                          lse.data_ptr(), ws.data_ptr(), need, st))
    return o, lse


def attention_backward(q, k, v, o, lse, do, offsets=None, k_offsets=None, causal: bool = True, window: int = 0,
                       scale=None, stream=None):
    """Gradients of attention_forward from its inputs, its results and dL/do: {"dq", "dk",
    "dv"}, dense, in the activations' dtype."""
    if stream is not None:
        return _call_on(stream, attention_backward,
                        (q, k, v, o, lse, do, offsets, k_offsets, causal, window, scale))
    desc, views = _attention(q, k, v, offsets, k_offsets, causal, window, scale)
    dtype, dev = q.dtype, q.device
    oh, gh = _heads("o", o, q.shape, dtype, dev), _heads("do", do, q.shape, dtype, dev)
    _dense("lse", lse, (q.shape[1], q.shape[0]), torch.float32, dev)
    st = _on(dev)
    out = [torch.empty_like(t, memory_format=_DENSE) for t in (q, k, v)]
    ref = ctypes.byref(desc)
    need = load().ipttt_attention_backward_workspace_bytes(ref)
    ws = _temp(need, dev)
    _check(load().ipttt_attention_backward(
        ref, *views, oh, lse.data_ptr(), gh, *(_heads("out", t, t.shape, dtype, dev) for t in out), ws.data_ptr(),
        need, st))
    return dict(zip(("dq", "dk", "dv"), out))


def attention_step(q, cache, table, lens, window: int = 0, scale=None, stream=None):
    """Attention of one new token of each sequence over the cache: q [sequences, q_heads,
    head_dim], table int32 [sequences, pages], lens int32 [sequences], the keys of each
    sequence, the new token's own (appended before) among them. window > 0: the last
    `window` of them. Returns o like q, dense."""
    if stream is not None:
        return _call_on(stream, attention_step, (q, cache, table, lens, window, scale), (cache.k, cache.v))
    n, hq, dh = _three("q", q)
    dtype, dev = cache.dtype, cache.device
    qh = _heads("q", q, (n, hq, cache.head_dim), dtype, dev)
    tab = cache.table(table)
    if tab.batch != n:
        raise _invalid(f"table has {tab.batch} sequences, expected {n}")
    _dense("lens", lens, (n,), torch.int32, dev)
    st = _on(dev)
    o = torch.empty_like(q, memory_format=_DENSE)
    desc = ctypes.byref(StepDesc(hq, _int32("window", window), dh ** -0.5 if scale is None else scale))
    need = load().ipttt_attention_step_workspace_bytes(desc, cache._ref, tab)
    ws = _temp(need, dev)
    _check(load().ipttt_attention_step(desc, qh, cache._ref, tab, lens.data_ptr(),
                                       _heads("o", o, q.shape, dtype, dev), None, ws.data_ptr(), need, st))
    return o

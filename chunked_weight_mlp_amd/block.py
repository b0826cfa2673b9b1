"""The operators around the fast-weight layer (include/ipttt_block.h): layer norm,
the gated linear recurrence and the gated feed-forward block, forward and
backward, over libipttt's HIP kernels.

The `ipttt_*` functions are the C entry points with tensors for pointers; Norm
and FeedForward hold an operator's weights, and recurrence_forward / _step /
_backward allocate their outputs and workspace. Errors are ipttt.IptttError.
Tensors must be on the device of the stream the call runs on (`stream`, or the
current one); a stream other than the current one must already be ordered after
whatever produced the inputs, as with any torch tensor.
"""
from __future__ import annotations

import ctypes

import torch

from . import ipttt as _b
from .ipttt import IPTTT_E_INVALID, IPTTT_E_UNSUPPORTED, IptttError, _check, _stream

_DT = _b._DT

EXPORTS = (
    "ipttt_norm_forward", "ipttt_norm_backward_workspace_bytes", "ipttt_norm_backward",
    "ipttt_recurrence_workspace_bytes", "ipttt_recurrence_forward", "ipttt_recurrence_step",
    "ipttt_recurrence_backward", "ipttt_ff_workspace_bytes", "ipttt_ff_forward",
    "ipttt_ff_backward_workspace_bytes", "ipttt_ff_backward",
)


class NormDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class View(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("tok_stride", ctypes.c_int64)]


class RecurrenceDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("d", ctypes.c_int32), ("seq_len", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("g", View), ("v", View), ("h", View),
                ("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("h0", ctypes.c_void_p)]


class FFDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p)]


class FFGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_int64),
                ("dw_gate", ctypes.c_void_p), ("dw_up", ctypes.c_void_p),
                ("dw_down", ctypes.c_void_p)]


_lib = None


def load() -> ctypes.CDLL:
    """The library with this header's signatures; raises if it is not built."""
    global _lib
    if _lib is None:
        lib = _b.load()
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        sig = {
            "ipttt_norm_forward": [P(NormDesc), vp, i64, vp, i64, i64, vp, vp, vp, vp, vp],
            "ipttt_norm_backward": [P(NormDesc), vp, i64, vp, vp, vp, i64, vp, i64, i64, vp, vp, vp,
                                    vp, sz, vp],
            "ipttt_recurrence_forward": [P(RecurrenceDesc), vp, vp, sz, vp],
            "ipttt_recurrence_step": [P(RecurrenceDesc), vp, vp],
            "ipttt_recurrence_backward": [P(RecurrenceDesc), P(View), vp, P(View), P(View), vp, vp,
                                          sz, vp],
            "ipttt_ff_forward": [P(FFDesc), vp, i64, i64, vp, i64, vp, vp, vp, sz, vp],
            "ipttt_ff_backward": [P(FFDesc), vp, i64, vp, vp, vp, i64, i64, P(FFGrads), vp, sz, vp],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        for name, args in {"ipttt_norm_backward_workspace_bytes": [P(NormDesc), i64],
                           "ipttt_recurrence_workspace_bytes": [P(RecurrenceDesc)],
                           "ipttt_ff_workspace_bytes": [P(FFDesc), i64],
                           "ipttt_ff_backward_workspace_bytes": [P(FFDesc), i64]}.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, sz
        _lib = lib
    return _lib


# ---- the C entry points -----------------------------------------------------------------


def _p(t):
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _ref(s):
    return None if s is None else ctypes.byref(s)


def ipttt_norm_forward(desc, x, x_stride, r, r_stride, n, h, y, mean, rstd, stream=None) -> None:
    _check(load().ipttt_norm_forward(_ref(desc), _p(x), x_stride, _p(r), r_stride, n, _p(h), _p(y),
                                     _p(mean), _p(rstd), _stream(stream)))


def ipttt_norm_backward_workspace_bytes(desc, n: int) -> int:
    return load().ipttt_norm_backward_workspace_bytes(_ref(desc), n)


def ipttt_norm_backward(desc, h, h_stride, mean, rstd, dy, dy_stride, dh, dh_stride, n, dx, dgamma,
                        dbeta, workspace, workspace_bytes, stream=None) -> None:
    _check(load().ipttt_norm_backward(_ref(desc), _p(h), h_stride, _p(mean), _p(rstd), _p(dy),
                                      dy_stride, _p(dh), dh_stride, n, _p(dx), _p(dgamma), _p(dbeta),
                                      _p(workspace), workspace_bytes, _stream(stream)))


def ipttt_recurrence_workspace_bytes(desc) -> int:
    return load().ipttt_recurrence_workspace_bytes(_ref(desc))


def ipttt_recurrence_forward(desc, h_last, workspace, workspace_bytes, stream=None) -> None:
    _check(load().ipttt_recurrence_forward(_ref(desc), _p(h_last), _p(workspace), workspace_bytes,
                                           _stream(stream)))


def ipttt_recurrence_step(desc, state, stream=None) -> None:
    _check(load().ipttt_recurrence_step(_ref(desc), _p(state), _stream(stream)))


def ipttt_recurrence_backward(desc, dh, dh_last, dg, dv, dh0, workspace, workspace_bytes,
                              stream=None) -> None:
    _check(load().ipttt_recurrence_backward(_ref(desc), _ref(dh), _p(dh_last), _ref(dg), _ref(dv),
                                            _p(dh0), _p(workspace), workspace_bytes,
                                            _stream(stream)))


def ipttt_ff_workspace_bytes(desc, n: int) -> int:
    return load().ipttt_ff_workspace_bytes(_ref(desc), n)


def ipttt_ff_forward(desc, x, x_stride, n, y, y_stride, a, u, workspace, workspace_bytes,
                     stream=None) -> None:
    _check(load().ipttt_ff_forward(_ref(desc), _p(x), x_stride, n, _p(y), y_stride, _p(a), _p(u),
                                   _p(workspace), workspace_bytes, _stream(stream)))


def ipttt_ff_backward_workspace_bytes(desc, n: int) -> int:
    return load().ipttt_ff_backward_workspace_bytes(_ref(desc), n)


def ipttt_ff_backward(desc, x, x_stride, a, u, dy, dy_stride, n, grads, workspace, workspace_bytes,
                      stream=None) -> None:
    _check(load().ipttt_ff_backward(_ref(desc), _p(x), x_stride, _p(a), _p(u), _p(dy), dy_stride, n,
                                    _ref(grads), _p(workspace), workspace_bytes, _stream(stream)))


# ---- operators over tensors ---------------------------------------------------------------


def _invalid(msg: str) -> IptttError:
    return IptttError(IPTTT_E_INVALID, "IPTTT_E_INVALID: " + msg)


def _dtype_of(t):
    if t.dtype not in _DT:
        raise IptttError(IPTTT_E_UNSUPPORTED, f"IPTTT_E_UNSUPPORTED: dtype {t.dtype}")
    return _DT[t.dtype]


def _like(name, t, shape, dtype, device):
    """Checks a tensor's shape, type and device."""
    if tuple(t.shape) != tuple(shape):
        raise _invalid(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise _invalid(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise _invalid(f"{name} is on {t.device}, expected {device}")
    return t


def _dense(name, t, shape, dtype, device):
    _like(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise _invalid(f"{name} must be contiguous")
    return t


def _rows(name, t, d, dtype=None, device=None, n=None):
    """(row stride) of a tensor of rows [..., d]: [n, d] of any row stride, or any
    number of leading dimensions laid out as equally spaced rows."""
    if t.dim() < 1 or t.shape[-1] != d:
        raise _invalid(f"{name} has shape {tuple(t.shape)}, expected rows of {d}")
    if dtype is not None:
        _like(name, t, t.shape, dtype, device)
    rows = t.numel() // d
    if n is not None and rows != n:
        raise _invalid(f"{name} has {rows} rows, expected {n}")
    if rows > 0 and d > 1 and t.stride(-1) != 1:
        raise _invalid(f"{name} must have its last dimension contiguous")
    stride, span = d, 1
    first = True
    for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if first:
            stride, first = st, False
        elif st != stride * span:
            raise _invalid(f"{name}'s leading dimensions are not equally spaced rows")
        span *= size
    return stride


def _temp(nbytes, device, stream):
    """Workspace from torch's allocator. On a stream other than the current one the
    allocator is told, so the memory is not handed out again while the call runs."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _used_on(stream, t)
    return t


def _used_on(stream, *tensors):
    if stream is None:
        return
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    if stream != torch.cuda.current_stream(stream.device):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)


class Norm:
    """Layer norm over rows of d, with the residual add in front of it. gamma, beta:
    [d] in the activations' dtype (float32 or bfloat16), beta may be None."""

    def __init__(self, gamma, beta=None, eps: float = 1e-5):
        if gamma.dim() != 1:
            raise _invalid("gamma must be [d]")
        self.d, self.dtype, self.device = gamma.shape[0], gamma.dtype, gamma.device
        dt = _dtype_of(gamma)
        self.gamma = _dense("gamma", gamma, (self.d,), self.dtype, self.device)
        self.beta = None if beta is None else _dense("beta", beta, (self.d,), self.dtype, self.device)
        self.desc = NormDesc(d=self.d, dtype=dt, eps=eps, gamma=_p(gamma), beta=_p(beta))

    def forward(self, x, res=None, stream=None):
        """Returns (y, h, mean, rstd): h = x + res (x itself without res), y its norm,
        and the rows' statistics for the backward. x, res: [..., d]."""
        xs = _rows("x", x, self.d, self.dtype, self.device)
        lead = x.shape[:-1]
        n = x.numel() // self.d
        y = torch.empty(x.shape, dtype=self.dtype, device=self.device)
        stats = torch.empty((2,) + tuple(lead), dtype=torch.float32, device=self.device)
        mean, rstd = stats[0], stats[1]
        rs, h = 0, None
        if res is not None:
            rs = _rows("res", res, self.d, self.dtype, self.device, n)
            h = torch.empty(x.shape, dtype=self.dtype, device=self.device)
        ipttt_norm_forward(self.desc, x, xs, res, rs, n, h, y, mean, rstd, stream)
        _used_on(stream, x, res, h, y, stats, self.gamma, self.beta)
        return y, (x if h is None else h), mean, rstd

    def backward(self, h, mean, rstd, dy, dh=None, stream=None):
        """Returns {"dx", "dgamma", "dbeta"}: the gradient of x and res ([..., d], the
        activations' dtype) and the fp32 weight gradients, from dL/dy and dL/dh."""
        hs = _rows("h", h, self.d, self.dtype, self.device)
        n = h.numel() // self.d
        ds = _rows("dy", dy, self.d, self.dtype, self.device, n)
        hh = 0 if dh is None else _rows("dh", dh, self.d, self.dtype, self.device, n)
        for name, t in (("mean", mean), ("rstd", rstd)):
            if t.numel() != n:
                raise _invalid(f"{name} has {t.numel()} values, expected {n}")
            _dense(name, t, t.shape, torch.float32, self.device)
        dx = torch.empty(h.shape, dtype=self.dtype, device=self.device)
        sums = torch.empty((2, self.d), dtype=torch.float32, device=self.device)
        need = ipttt_norm_backward_workspace_bytes(self.desc, n)
        ws = _temp(need, self.device, stream)
        ipttt_norm_backward(self.desc, h, hs, mean, rstd, dy, ds, dh, hh, n, dx, sums[0], sums[1],
                            ws, need, stream)
        _used_on(stream, h, mean, rstd, dy, dh, dx, sums, self.gamma)
        return {"dx": dx, "dgamma": sums[0], "dbeta": sums[1]}


def _view(name, t, shape, dtype, device):
    _like(name, t, shape, dtype, device)
    if t.numel() and shape[2] > 1 and t.stride(2) != 1:
        raise _invalid(f"{name} must have its channels contiguous")
    return View(p=t.data_ptr(), seq_stride=t.stride(0), tok_stride=t.stride(1))


def _recurrence(g, v, h, h0, starts, lens):
    if g.dim() != 3:
        raise _invalid("g must be [batch, seq_len, d]")
    n, length, d = g.shape
    dev = g.device
    r = RecurrenceDesc(batch=n, d=d, seq_len=length, dtype=_dtype_of(g))
    r.g = _view("g", g, g.shape, g.dtype, dev)
    r.v = _view("v", v, g.shape, g.dtype, dev)
    r.h = _view("h", h, g.shape, g.dtype, dev)
    if h0 is not None:
        r.h0 = _p(_dense("h0", h0, (n, d), torch.float32, dev))
    if starts is not None:
        if starts.dtype == torch.bool:
            starts = starts.view(torch.uint8)
        r.starts = _p(_dense("starts", starts, (n, length), torch.uint8, dev))
    if lens is not None:
        r.lens = _p(_dense("lens", lens, (n,), torch.int32, dev))
    return r


def recurrence_forward(g, v, h0=None, starts=None, lens=None, stream=None):
    """h_t = f_t h_{t-1} + (1 - f_t) v_t with f = sigmoid(g), for g, v [batch, seq_len, d]
    (slices of a wider tensor will do). h0: fp32 [batch, d]; starts: bool or uint8
    [batch, seq_len], nonzero where a packed document begins; lens: int32 [batch].
    Returns (h, h_last): h like g, h_last fp32 [batch, d], the state for the next call."""
    h = torch.empty(g.shape, dtype=g.dtype, device=g.device)
    r = _recurrence(g, v, h, h0, starts, lens)
    last = torch.empty((r.batch, r.d), dtype=torch.float32, device=g.device)
    need = ipttt_recurrence_workspace_bytes(r)
    ws = _temp(need, g.device, stream)
    ipttt_recurrence_forward(r, last, ws, need, stream)
    _used_on(stream, g, v, h0, starts, lens, h, last)
    return h, last


def recurrence_step(g, v, state, out=None, stream=None):
    """One token per sequence: g, v [batch, d], state fp32 [batch, d] or None (zero).
    Returns (h [batch, d], the new state); pass out=state to update it in place."""
    if g.dim() != 2:
        raise _invalid("g must be [batch, d]")
    h = torch.empty(g.shape, dtype=g.dtype, device=g.device)
    r = _recurrence(g.unsqueeze(1), v.unsqueeze(1), h.unsqueeze(1), state, None, None)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.float32, device=g.device)
    else:
        _dense("out", out, g.shape, torch.float32, g.device)
    ipttt_recurrence_step(r, out, stream)
    _used_on(stream, g, v, state, h, out)
    return h, out


def recurrence_backward(g, v, h, dh, h0=None, dh_last=None, starts=None, lens=None, dg=None, dv=None,
                        stream=None):
    """Gradients of recurrence_forward from its output h, dL/dh and dL/dh_last (fp32
    [batch, d] or None): {"dg", "dv", "dh0"}. dg and dv may be passed in (for
    example the two halves of one projection's gradient)."""
    r = _recurrence(g, v, h, h0, starts, lens)
    dev = g.device
    dg = torch.empty(g.shape, dtype=g.dtype, device=dev) if dg is None else dg
    dv = torch.empty(g.shape, dtype=g.dtype, device=dev) if dv is None else dv
    dh0 = torch.empty((r.batch, r.d), dtype=torch.float32, device=dev)
    if dh_last is not None:
        _dense("dh_last", dh_last, (r.batch, r.d), torch.float32, dev)
    need = ipttt_recurrence_workspace_bytes(r)
    ws = _temp(need, dev, stream)
    ipttt_recurrence_backward(r, _view("dh", dh, g.shape, g.dtype, dev), dh_last,
                              _view("dg", dg, g.shape, g.dtype, dev),
                              _view("dv", dv, g.shape, g.dtype, dev), dh0, ws, need, stream)
    _used_on(stream, g, v, h, dh, h0, dh_last, starts, lens, dg, dv, dh0)
    return {"dg": dg, "dv": dv, "dh0": dh0}


class FeedForward:
    """The gated feed-forward block y = (SiLU(x W_g) * (x W_u)) W_d with output-major
    weights: w_gate, w_up [d_ff, d], w_down [d, d_ff], float32 or bfloat16."""

    def __init__(self, w_gate, w_up, w_down):
        if w_gate.dim() != 2:
            raise _invalid("w_gate must be [d_ff, d]")
        f, d = w_gate.shape
        self.d, self.d_ff, self.dtype, self.device = d, f, w_gate.dtype, w_gate.device
        dt = _dtype_of(w_gate)
        self.w_gate = _dense("w_gate", w_gate, (f, d), self.dtype, self.device)
        self.w_up = _dense("w_up", w_up, (f, d), self.dtype, self.device)
        self.w_down = _dense("w_down", w_down, (d, f), self.dtype, self.device)
        self.desc = FFDesc(d=d, d_ff=f, dtype=dt, w_gate=_p(w_gate), w_up=_p(w_up), w_down=_p(w_down))

    def forward(self, x, save: bool = False, stream=None):
        """x: [..., d]. Returns y, or (y, a, u) with the pre-activations for the backward."""
        xs = _rows("x", x, self.d, self.dtype, self.device)
        n = x.numel() // self.d
        y = torch.empty(x.shape, dtype=self.dtype, device=self.device)
        a = u = None
        if save:
            a = torch.empty(x.shape[:-1] + (self.d_ff,), dtype=self.dtype, device=self.device)
            u = torch.empty_like(a)
        need = ipttt_ff_workspace_bytes(self.desc, n)
        ws = _temp(need, self.device, stream)
        ipttt_ff_forward(self.desc, x, xs, n, y, self.d, a, u, ws, need, stream)
        _used_on(stream, x, y, a, u, self.w_gate, self.w_up, self.w_down)
        return (y, a, u) if save else y

    def backward(self, x, a, u, dy, stream=None):
        """Gradients from dL/dy and the saved pre-activations: {"dx", "dw_gate", "dw_up",
        "dw_down"}, all in the weights' dtype."""
        xs = _rows("x", x, self.d, self.dtype, self.device)
        n = x.numel() // self.d
        ds = _rows("dy", dy, self.d, self.dtype, self.device, n)
        for name, t in (("a", a), ("u", u)):
            _dense(name, t, x.shape[:-1] + (self.d_ff,), self.dtype, self.device)
        new = lambda s: torch.empty(s, dtype=self.dtype, device=self.device)  # noqa: E731
        g = {"dx": new(x.shape), "dw_gate": new((self.d_ff, self.d)), "dw_up": new((self.d_ff, self.d)),
             "dw_down": new((self.d, self.d_ff))}
        need = ipttt_ff_backward_workspace_bytes(self.desc, n)
        ws = _temp(need, self.device, stream)
        ipttt_ff_backward(self.desc, x, xs, a, u, dy, ds, n,
                          FFGrads(dx_stride=self.d, **{k: _p(t) for k, t in g.items()}), ws, need,
                          stream)
        _used_on(stream, x, a, u, dy, self.w_gate, self.w_up, self.w_down, *g.values())
        return g

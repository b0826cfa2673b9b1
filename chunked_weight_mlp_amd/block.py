"""The operators around the fast-weight layer (include/ipttt_block.h): layer norm,
the gated linear recurrence and the gated feed-forward block, forward and
backward, over libipttt's HIP kernels.

The `ipttt_*` functions are the C entry points with tensors for pointers; Norm
and FeedForward hold an operator's weights, and recurrence_forward / _step /
_backward allocate their outputs and workspace. Errors are ipttt.IptttError.
Tensors must be on the device of the stream the call runs on: the current one, or
`stream` (a torch stream or its handle), with which a call does what it would do
under `torch.cuda.stream(stream)`: its outputs and workspace come from that stream's
memory. Such a stream must already be ordered after whatever produced the inputs, and
whoever uses the outputs on another stream after this one, as with any torch tensor;
that neither's memory is handed out again too early, on `stream` or on the stream
that was current, is taken care of.

Outputs are detached: the operators record nothing for torch's autograd, and an input
that requires a gradient is used by its value. Their `backward` calls give the gradients.
"""
from __future__ import annotations

import ctypes

import torch

from . import ipttt as _b
from .ipttt import IPTTT_E_INVALID, IPTTT_E_UNSUPPORTED, IptttError, _check, _stream

_DT = _b._DT
_DENSE = torch.contiguous_format

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


class _FlatRecurrence(ctypes.Structure):
    """RecurrenceDesc with its views' fields side by side: the same layout, built in one call."""
    _fields_ = [("batch", ctypes.c_int32), ("d", ctypes.c_int32), ("seq_len", ctypes.c_int64),
                ("dtype", ctypes.c_int)] + [
        (f"{v}_{f}", t) for v in "gvh"
        for f, t in (("p", ctypes.c_void_p), ("seq", ctypes.c_int64), ("tok", ctypes.c_int64))] + [
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
            "ipttt_recurrence_forward": [vp, vp, vp, sz, vp],
            "ipttt_recurrence_step": [vp, vp, vp],
            "ipttt_recurrence_backward": [vp, P(View), vp, P(View), P(View), vp, vp,
                                          sz, vp],
            "ipttt_ff_forward": [P(FFDesc), vp, i64, i64, vp, i64, vp, vp, vp, sz, vp],
            "ipttt_ff_backward": [P(FFDesc), vp, i64, vp, vp, vp, i64, i64, P(FFGrads), vp, sz, vp],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        for name, args in {"ipttt_norm_backward_workspace_bytes": [P(NormDesc), i64],
                           "ipttt_recurrence_workspace_bytes": [vp],
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
    dt = _DT.get(t.dtype)
    if dt is None:
        raise IptttError(IPTTT_E_UNSUPPORTED, f"IPTTT_E_UNSUPPORTED: dtype {t.dtype}")
    return dt


def _is(name, t, dtype, device):
    """Checks a tensor's type and device."""
    if t.dtype is not dtype:
        raise _invalid(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise _invalid(f"{name} is on {t.device}, expected {device}")


def _dense(name, t, shape, dtype, device):
    if t.shape != shape:
        raise _invalid(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _is(name, t, dtype, device)
    if not t.is_contiguous():
        raise _invalid(f"{name} must be contiguous")
    return t


def _rows(name, t, d, dtype, device, n=None):
    """The row stride of a tensor of rows [..., d]: [n, d] of any row stride, or any
    number of leading dimensions laid out as equally spaced rows."""
    shape = t.shape
    if (t.dtype is dtype and t.device == device and shape and shape[-1] == d and t.is_contiguous()
            and (n is None or t.numel() == n * d)):
        return d
    if not shape or shape[-1] != d:
        raise _invalid(f"{name} has shape {tuple(shape)}, expected rows of {d}")
    _is(name, t, dtype, device)
    rows = t.numel() // d
    if n is not None and rows != n:
        raise _invalid(f"{name} has {rows} rows, expected {n}")
    if rows > 0 and d > 1 and t.stride(-1) != 1:
        raise _invalid(f"{name} must have its last dimension contiguous")
    stride, span, first = d, 1, True
    for size, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if first:
            stride, first = st, False
        elif st != stride * span:
            raise _invalid(f"{name}'s leading dimensions are not equally spaced rows")
        span *= size
    return stride


# The current stream's handle without building a torch.cuda.Stream for it, which
# takes about as long as a small kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(device):
    """The current HIP stream, for a call whose tensors are on `device`."""
    index = device.index
    if device.type != "cuda":
        raise _invalid(f"tensors are on {device}, not on a GPU")
    if index != torch.cuda.current_device():
        raise _invalid(f"tensors are on {device}, the current device is cuda:"
                       f"{torch.cuda.current_device()}")
    return _stream(None) if _raw_stream is None else _raw_stream(index)


def _call_on(stream, op, args, weights=()):
    """op(*args) on another stream than the current one. Outputs and workspace are
    allocated as that stream's: a block of the current stream's memory may still have
    work queued on it by a tensor that is gone, which `stream` is not ordered after.
    The allocator is told that `stream` uses the inputs, and the current stream the
    outputs, so that neither is handed out again while the other still works on it."""
    if args[0].device.type != "cuda":
        return op(*args)   # which refuses them
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return op(*args)
    with torch.cuda.stream(stream):
        out = op(*args)
    for t in (*args, *weights):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    for t in (out,) if isinstance(out, torch.Tensor) else out.values() if isinstance(out, dict) else out:
        if t is not None:
            t.record_stream(current)
    return out


def _temp(nbytes, device):
    """Workspace from torch's allocator."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


class Norm:
    """Layer norm over rows of d, with the residual add in front of it. gamma, beta:
    [d] in the activations' dtype (float32 or bfloat16), beta may be None."""

    def __init__(self, gamma, beta=None, eps: float = 1e-5):
        if gamma.dim() != 1 or gamma.numel() == 0:
            raise _invalid("gamma must be [d], d > 0")
        self.d, self.dtype, self.device = gamma.shape[0], gamma.dtype, gamma.device
        dt = _dtype_of(gamma)
        self.gamma = _dense("gamma", gamma, (self.d,), self.dtype, self.device)
        self.beta = None if beta is None else _dense("beta", beta, (self.d,), self.dtype, self.device)
        self.desc = NormDesc(d=self.d, dtype=dt, eps=eps, gamma=_p(gamma), beta=_p(beta))
        self._ref = ctypes.byref(self.desc)

    def forward(self, x, res=None, stream=None):
        """Returns (y, h, mean, rstd): h = x + res (x itself without res), y its norm,
        and the rows' statistics for the backward. x, res: [..., d]."""
        if stream is not None:
            return _call_on(stream, self.forward, (x, res), (self.gamma, self.beta))
        d, dtype, dev = self.d, self.dtype, self.device
        xs = _rows("x", x, d, dtype, dev)
        st = _on(dev)
        shape = x.shape
        n = x.numel() // d
        y = torch.empty_like(x, memory_format=_DENSE)
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        r = hp = h = None
        rs = 0
        if res is not None:
            rs, r = _rows("res", res, d, dtype, dev, n), res.data_ptr()
            h = torch.empty_like(x, memory_format=_DENSE)
            hp = h.data_ptr()
        _check(load().ipttt_norm_forward(self._ref, x.data_ptr(), xs, r, rs, n, hp, y.data_ptr(),
                                         mean.data_ptr(), rstd.data_ptr(), st))
        return y, (x if h is None else h), mean, rstd

    def backward(self, h, mean, rstd, dy, dh=None, stream=None):
        """Returns {"dx", "dgamma", "dbeta"}: the gradient of x and res ([..., d], the
        activations' dtype) and the fp32 weight gradients, from dL/dy and dL/dh."""
        if stream is not None:
            return _call_on(stream, self.backward, (h, mean, rstd, dy, dh), (self.gamma,))
        d, dtype, dev = self.d, self.dtype, self.device
        hs = _rows("h", h, d, dtype, dev)
        st = _on(dev)
        n = h.numel() // d
        ds = _rows("dy", dy, d, dtype, dev, n)
        hh = 0 if dh is None else _rows("dh", dh, d, dtype, dev, n)
        for name, t in (("mean", mean), ("rstd", rstd)):
            if t.numel() != n:
                raise _invalid(f"{name} has {t.numel()} values, expected {n}")
            if t.dtype is not torch.float32 or t.device != dev or not t.is_contiguous():
                _dense(name, t, t.shape, torch.float32, dev)
        dx = torch.empty_like(h, memory_format=_DENSE)
        dgamma = torch.empty(d, dtype=torch.float32, device=dev)
        dbeta = torch.empty(d, dtype=torch.float32, device=dev)
        need = load().ipttt_norm_backward_workspace_bytes(self._ref, n)
        ws = _temp(need, dev)
        _check(load().ipttt_norm_backward(self._ref, h.data_ptr(), hs, mean.data_ptr(), rstd.data_ptr(),
                                          dy.data_ptr(), ds, _p(dh), hh, n, dx.data_ptr(),
                                          dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), need, st))
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _strides(name, t, shape, dtype, device):
    """(pointer, sequence stride, token stride) of a [batch, seq_len, d] tensor, or of
    [batch, d] as one token each."""
    if t.shape != shape:
        raise _invalid(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        _is(name, t, dtype, device)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1 and t.numel():
        raise _invalid(f"{name} must have its channels contiguous")
    return t.data_ptr(), stride[0], stride[-2]


def _recurrence(g, v, h, h0, starts=None, lens=None):
    shape, dtype, dev = g.shape, g.dtype, g.device
    n, d = shape[0], shape[-1]
    length = shape[1] if len(shape) == 3 else 1
    dt = _dtype_of(g)
    if h0 is not None:
        h0 = _dense("h0", h0, (n, d), torch.float32, dev).data_ptr()
    if starts is not None:
        if starts.dtype is torch.bool:
            starts = starts.view(torch.uint8)
        starts = _dense("starts", starts, (n, length), torch.uint8, dev).data_ptr()
    if lens is not None:
        lens = _dense("lens", lens, (n,), torch.int32, dev).data_ptr()
    return _FlatRecurrence(n, d, length, dt, *_strides("g", g, shape, dtype, dev),
                           *_strides("v", v, shape, dtype, dev), *_strides("h", h, shape, dtype, dev),
                           starts, lens, h0)


def recurrence_forward(g, v, h0=None, starts=None, lens=None, stream=None):
    """h_t = f_t h_{t-1} + (1 - f_t) v_t with f = sigmoid(g), for g, v [batch, seq_len, d]
    (slices of a wider tensor will do). h0: fp32 [batch, d]; starts: bool or uint8
    [batch, seq_len], nonzero where a packed document begins; lens: int32 [batch].
    Returns (h, h_last): h like g, h_last fp32 [batch, d], the state for the next call."""
    if stream is not None:
        return _call_on(stream, recurrence_forward, (g, v, h0, starts, lens))
    if g.dim() != 3:
        raise _invalid("g must be [batch, seq_len, d]")
    dev = g.device
    st = _on(dev)
    h = torch.empty_like(g, memory_format=_DENSE)
    r = _recurrence(g, v, h, h0, starts, lens)
    last = torch.empty((r.batch, r.d), dtype=torch.float32, device=dev)
    ref = ctypes.byref(r)
    need = load().ipttt_recurrence_workspace_bytes(ref)
    ws = _temp(need, dev)
    _check(load().ipttt_recurrence_forward(ref, last.data_ptr(), ws.data_ptr(), need, st))
    return h, last


def recurrence_step(g, v, state, out=None, stream=None):
    """One token per sequence: g, v [batch, d], state fp32 [batch, d] or None (zero).
    Returns (h [batch, d], the new state); pass out=state to update it in place."""
    if stream is not None:
        return _call_on(stream, recurrence_step, (g, v, state, out))
    if g.dim() != 2:
        raise _invalid("g must be [batch, d]")
    dev = g.device
    st = _on(dev)
    h = torch.empty_like(g, memory_format=_DENSE)
    r = _recurrence(g, v, h, state)
    if out is None:
        out = (torch.empty_like(state) if state is not None else
               torch.empty(g.shape, dtype=torch.float32, device=dev))
    else:
        _dense("out", out, g.shape, torch.float32, dev)
    _check(load().ipttt_recurrence_step(ctypes.byref(r), out.data_ptr(), st))
    return h, out


def recurrence_backward(g, v, h, dh, h0=None, dh_last=None, starts=None, lens=None, dg=None, dv=None,
                        stream=None):
    """Gradients of recurrence_forward from its output h, dL/dh and dL/dh_last (fp32
    [batch, d] or None): {"dg", "dv", "dh0"}. dg and dv may be passed in (for
    example the two halves of one projection's gradient); they must overlap neither
    each other nor an input."""
    if stream is not None:
        return _call_on(stream, recurrence_backward, (g, v, h, dh, h0, dh_last, starts, lens, dg, dv))
    if g.dim() != 3:
        raise _invalid("g must be [batch, seq_len, d]")
    shape, dtype, dev = g.shape, g.dtype, g.device
    st = _on(dev)
    r = _recurrence(g, v, h, h0, starts, lens)
    dg = torch.empty_like(g, memory_format=_DENSE) if dg is None else dg
    dv = torch.empty_like(g, memory_format=_DENSE) if dv is None else dv
    dh0 = torch.empty((r.batch, r.d), dtype=torch.float32, device=dev)
    if dh_last is not None:
        _dense("dh_last", dh_last, (r.batch, r.d), torch.float32, dev)
    views = [ctypes.byref(View(*_strides(name, t, shape, dtype, dev)))
             for name, t in (("dh", dh), ("dg", dg), ("dv", dv))]
    ref = ctypes.byref(r)
    need = load().ipttt_recurrence_workspace_bytes(ref)
    ws = _temp(need, dev)
    _check(load().ipttt_recurrence_backward(ref, views[0], _p(dh_last), views[1], views[2],
                                            dh0.data_ptr(), ws.data_ptr(), need, st))
    return {"dg": dg, "dv": dv, "dh0": dh0}


class FeedForward:
    """The gated feed-forward block y = (SiLU(x W_g) * (x W_u)) W_d with output-major
    weights: w_gate, w_up [d_ff, d], w_down [d, d_ff], float32 or bfloat16."""

    def __init__(self, w_gate, w_up, w_down):
        if w_gate.dim() != 2 or w_gate.numel() == 0:
            raise _invalid("w_gate must be [d_ff, d], both > 0")
        f, d = w_gate.shape
        self.d, self.d_ff, self.dtype, self.device = d, f, w_gate.dtype, w_gate.device
        dt = _dtype_of(w_gate)
        self.w_gate = _dense("w_gate", w_gate, (f, d), self.dtype, self.device)
        self.w_up = _dense("w_up", w_up, (f, d), self.dtype, self.device)
        self.w_down = _dense("w_down", w_down, (d, f), self.dtype, self.device)
        self.desc = FFDesc(d=d, d_ff=f, dtype=dt, w_gate=_p(w_gate), w_up=_p(w_up), w_down=_p(w_down))
        self._ref = ctypes.byref(self.desc)

    def forward(self, x, save: bool = False, stream=None):
        """x: [..., d]. Returns y, or (y, a, u) with the pre-activations (fp32) for the
        backward."""
        if stream is not None:
            return _call_on(stream, self.forward, (x, save), (self.w_gate, self.w_up, self.w_down))
        d, dtype, dev = self.d, self.dtype, self.device
        xs = _rows("x", x, d, dtype, dev)
        st = _on(dev)
        n = x.numel() // d
        y = torch.empty_like(x, memory_format=_DENSE)
        a = u = None
        if save:
            a = torch.empty(x.shape[:-1] + (self.d_ff,), dtype=torch.float32, device=dev)
            u = torch.empty_like(a)
        need = load().ipttt_ff_workspace_bytes(self._ref, n)
        ws = _temp(need, dev)
        _check(load().ipttt_ff_forward(self._ref, x.data_ptr(), xs, n, y.data_ptr(), d, _p(a), _p(u),
                                       ws.data_ptr(), need, st))
        return (y, a, u) if save else y

    def backward(self, x, a, u, dy, stream=None):
        """Gradients from dL/dy and the saved pre-activations: {"dx", "dw_gate", "dw_up",
        "dw_down"}, all in the weights' dtype."""
        if stream is not None:
            return _call_on(stream, self.backward, (x, a, u, dy), (self.w_gate, self.w_up, self.w_down))
        d, f, dtype, dev = self.d, self.d_ff, self.dtype, self.device
        xs = _rows("x", x, d, dtype, dev)
        st = _on(dev)
        n = x.numel() // d
        ds = _rows("dy", dy, d, dtype, dev, n)
        for name, t in (("a", a), ("u", u)):
            _dense(name, t, x.shape[:-1] + (f,), torch.float32, dev)
        dx = torch.empty_like(x, memory_format=_DENSE)
        dwg, dwu, dwd = (torch.empty_like(w) for w in (self.w_gate, self.w_up, self.w_down))
        need = load().ipttt_ff_backward_workspace_bytes(self._ref, n)
        ws = _temp(need, dev)
        grads = FFGrads(dx.data_ptr(), d, dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr())
        _check(load().ipttt_ff_backward(self._ref, x.data_ptr(), xs, a.data_ptr(), u.data_ptr(),
                                        dy.data_ptr(), ds, n, ctypes.byref(grads), ws.data_ptr(), need, st))
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}

"""The feed-forward operators on torch tensors: argument checks, outputs and
workspaces around the C ABI's ``tgemm_layer_norm``, ``tgemm_ffn_*``,
``tgemm_dropout`` and their backward passes.

Every function enqueues on torch's current stream and returns at once.  With
``stream`` it runs on that stream instead: outputs and workspaces are then
allocated for it, and the inputs are kept from reuse until it has passed the
call; ordering it after the inputs' producers stays with the caller.
"""

from __future__ import annotations

import ctypes
import threading

import software_pipelined_tiled_02_gb300 as _tg

# Filled on first use (torch is imported late), the library last: torch, its
# dtypes' codes, and the loaded library.
_torch = _CODES = _L = None


def _setup():
    global _torch, _CODES, _L
    import torch

    _torch = torch
    _CODES = {torch.float16: _tg.F16, torch.bfloat16: _tg.BF16, torch.float32: _tg.F32}
    _L = _tg.load()
    return _L


def _on_stream(stream, function, *args, **kwargs):
    """function(*args, **kwargs) with `stream` as the current stream."""
    if _L is None:
        _setup()
    with _torch.cuda.stream(stream):
        result = function(*args, **kwargs)
    for t in list(args) + list(kwargs.values()):
        for x in t if isinstance(t, (tuple, list)) else (t,):
            if isinstance(x, _torch.Tensor) and x.is_cuda:
                x.record_stream(stream)
    return result


# The checks below run on every call, so a message is only formed once a check
# has failed.

def _stream_ptr(index):
    # what torch.cuda.current_stream(index).cuda_stream is, without the Stream object (2.9 us of a call)
    return _torch._C._cuda_getCurrentRawStream(index)


def _tensor(name, t):
    """The index of the CUDA device tensor `t` lives on, which has to be the current one."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    index = t.get_device()
    if index != _torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return index


def _like(name, t, x, shape=True):
    """`t` has to be a tensor on x's device, of x's type and (by default) shape."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.device != x.device:
        raise ValueError(f"{name} must be on {x.device}, got {t.device}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, got {t.dtype}")
    if shape and t.shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}, got {tuple(t.shape)}")


def _code(name, t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be fp16, bf16 or fp32, got {t.dtype}")
    return code


def _row_width(x):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have a last dimension of at least 1, got {tuple(x.shape)}")
    return x.shape[-1]


def _rows(name, t, width):
    """(rows, elements from one row to the next) of a tensor whose last dimension holds rows of `width`."""
    if t.is_contiguous():
        return t.numel() // width, width
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous, or a matrix with contiguous rows")
    rows, ld = t.shape[0], t.stride(0)
    if rows <= 1:
        return rows, width
    if ld < width:
        raise ValueError(f"the rows of {name} must not overlap")
    return rows, ld


def _vector(name, t, width, x):
    """A weight vector's type code: x's type or fp32."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.device != x.device:
        raise ValueError(f"{name} must be on {x.device}, got {t.device}")
    if t.dim() != 1 or t.shape[0] != width or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape ({width},), got {tuple(t.shape)}")
    if t.dtype != x.dtype and t.dtype != _torch.float32:
        raise TypeError(f"{name} must be {x.dtype} or torch.float32, got {t.dtype}")
    return _CODES[t.dtype]


def layer_norm(x, weight=None, bias=None, eps=1e-5, stats=False, stream=None):
    """``(x - mean) / sqrt(var + eps) * weight + bias`` over the last dimension of x.

    x is fp16, bf16 or fp32: contiguous, or a matrix with contiguous rows.
    weight and bias (or None) share one type, x's or fp32.  With ``stats`` the
    result is ``(y, mean, rstd)``; mean and rstd are fp32, one value a row, as
    `layer_norm_backward` takes them.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, eps, stats)
    L = _L or _setup()
    index = _tensor("x", x)
    code = wcode = _code("x", x)
    width = _row_width(x)
    rows, ld = _rows("x", x, width)
    if weight is not None:
        wcode = _vector("weight", weight, width, x)
    if bias is not None:
        bcode = _vector("bias", bias, width, x)
        if weight is not None and bcode != wcode:
            raise TypeError(f"weight and bias must have the same type, got {weight.dtype} and {bias.dtype}")
        wcode = bcode
    device = x.device
    y = _torch.empty(x.shape, dtype=x.dtype, device=device)
    mean = _torch.empty(rows, dtype=_torch.float32, device=device) if stats else None
    rstd = _torch.empty(rows, dtype=_torch.float32, device=device) if stats else None
    rc = L.tgemm_layer_norm(
        rows, width, code, wcode, x.data_ptr(), ld, None if weight is None else weight.data_ptr(),
        None if bias is None else bias.data_ptr(), eps, y.data_ptr(), width, mean.data_ptr() if stats else None,
        rstd.data_ptr() if stats else None, _stream_ptr(index))
    if rc:
        raise _tg.TgemmError(rc, f"layer_norm(rows={rows}, width={width}, eps={eps})")
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, mean, rstd, weight=None, stream=None):
    """``(dx, dweight, dbias)`` of `layer_norm` from the gradient dy of its result.

    mean and rstd are what ``layer_norm(..., stats=True)`` returned.  dweight
    and dbias have weight's type, or x's without a weight.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, mean, rstd, weight)
    L = _L or _setup()
    index = _tensor("x", x)
    code = wcode = _code("x", x)
    width = _row_width(x)
    _like("dy", dy, x)
    rows, ldx = _rows("x", x, width)
    _, lddy = _rows("dy", dy, width)
    device = x.device
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != _torch.float32:
            raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
        if t.device != device or t.numel() != rows or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous on {device} with one value a row ({rows}), got {tuple(t.shape)}")
    wdtype = x.dtype
    if weight is not None:
        wcode, wdtype = _vector("weight", weight, width, x), weight.dtype
    dx = _torch.empty(x.shape, dtype=x.dtype, device=device)
    dw, db = _torch.empty(width, dtype=wdtype, device=device), _torch.empty(width, dtype=wdtype, device=device)
    need = L.tgemm_layer_norm_workspace(rows, width)
    if need < 0:
        raise _tg.TgemmError(-need, f"layer_norm_backward(rows={rows}, width={width})")
    work = _torch.empty(need, dtype=_torch.uint8, device=device)
    rc = L.tgemm_layer_norm_backward(
        rows, width, code, wcode, dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(),
        None if weight is None else weight.data_ptr(), dx.data_ptr(), width, dw.data_ptr(), db.data_ptr(),
        work.data_ptr(), need, _stream_ptr(index))
    if rc:
        raise _tg.TgemmError(rc, f"layer_norm_backward(rows={rows}, width={width})")
    return dx, dw, db


def dropout(x, p, seed, offset=0, residual=None, stream=None):
    """x with each element dropped with probability p, the others over 1 - p, plus residual.

    The mask is a function of (seed, offset) and the element's place alone
    (Philox4x32-10; include/tgemm.h has the layout), so `dropout_backward` with
    the same numbers meets the same mask.  seed and offset are taken modulo
    2^64; calls that share a seed take different offsets.
    """
    if stream is not None:
        return _on_stream(stream, dropout, x, p, seed, offset, residual)
    L = _L or _setup()
    index = _tensor("x", x)
    code = _code("x", x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if not 0 <= p <= 1:
        raise ValueError(f"p must lie between 0 and 1, got {p}")
    if residual is not None:
        _like("residual", residual, x)
        if not residual.is_contiguous():
            raise ValueError("residual must be contiguous")
    y = _torch.empty(x.shape, dtype=x.dtype, device=x.device)
    rc = L.tgemm_dropout(x.numel(), code, x.data_ptr(), None if residual is None else residual.data_ptr(),
                         y.data_ptr(), p, seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, _stream_ptr(index))
    if rc:
        raise _tg.TgemmError(rc, f"dropout(n={x.numel()}, p={p})")
    return y


def dropout_backward(dy, p, seed, offset=0, stream=None):
    """The gradient of `dropout`'s x (that of its residual is dy itself)."""
    return dropout(dy, p, seed, offset, stream=stream)


_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


class GatedFFN:
    """A plan of the gated feed-forward block ``y = (act(x Wg^T) * (x Wu^T)) Wd^T`` on the current device.

    x is a matrix [tokens, width] with any number of tokens, w_gate and w_up
    are [hidden, width], w_down is [width, hidden]; all fp16 or all bf16, rows
    contiguous and on 16-byte boundaries, width and hidden multiples of 8.
    activation: "silu", "gelu" (the exact one) or "relu".
    """

    def __init__(self, width, hidden, dtype="bf16", activation="silu"):
        self.handle = None
        L = _L or _setup()
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}, got {activation!r}")
        self.width, self.hidden, self.activation = int(width), int(hidden), activation
        self.dtype = _tg._dt(dtype)
        self.torch_dtype = _tg._torch_dtype(self.dtype)
        h = ctypes.c_void_p()
        rc = L.tgemm_ffn_plan(ctypes.byref(h), self.width, self.hidden, self.dtype, _ACTIVATIONS[activation])
        if rc:
            raise _tg.TgemmError(rc, f"tgemm_ffn_plan(width={width}, hidden={hidden}, activation={activation})")
        self.handle = h
        self.index = _torch.cuda.current_device()
        self.device = _torch.device("cuda", self.index)

    def _matrix(self, name, t, rows, cols):
        """Elements from row to row of a matrix argument."""
        if not isinstance(t, _torch.Tensor):
            raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
        if t.dtype != self.torch_dtype:
            raise TypeError(f"{name} must be {self.torch_dtype}, got {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        if t.shape != (rows, cols):
            raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
        if t.is_contiguous():
            return cols
        ld = t.stride(0) if rows > 1 else cols
        if t.stride(1) != 1 or ld < cols:
            raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
        return ld

    def forward(self, x, w_gate, w_up, w_down, save=False, stream=None):
        """y, or with ``save`` ``(y, (g, u, h))``: what `backward` takes."""
        if stream is not None:
            return _on_stream(stream, self.forward, x, w_gate, w_up, w_down, save)
        if x.dim() != 2:
            raise ValueError(f"x must be a matrix, got {tuple(x.shape)}")
        tokens, D, F, dtype, device = x.shape[0], self.width, self.hidden, self.torch_dtype, self.device
        m = self._matrix
        ldx, ldg, ldu, ldd = m("x", x, tokens, D), m("w_gate", w_gate, F, D), m("w_up", w_up, F, D), \
            m("w_down", w_down, D, F)
        y = _torch.empty((tokens, D), dtype=dtype, device=device)
        h = _torch.empty((tokens, F), dtype=dtype, device=device)
        g = _torch.empty((tokens, F), dtype=dtype, device=device) if save else None
        u = _torch.empty((tokens, F), dtype=dtype, device=device) if save else None
        rc = _L.tgemm_ffn_forward(
            self.handle, tokens, x.data_ptr(), ldx, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, w_down.data_ptr(), ldd,
            y.data_ptr(), D, g.data_ptr() if save else None, u.data_ptr() if save else None, h.data_ptr(),
            _stream_ptr(self.index))
        if rc:
            raise _tg.TgemmError(rc, f"tgemm_ffn_forward(tokens={tokens}, width={D}, hidden={F})")
        return (y, (g, u, h)) if save else y

    def backward(self, dy, x, w_gate, w_up, w_down, saved, stream=None):
        """``(dx, dw_gate, dw_up, dw_down)`` from the gradient dy of y and what ``forward(..., save=True)`` saved."""
        if stream is not None:
            return _on_stream(stream, self.backward, dy, x, w_gate, w_up, w_down, saved)
        if x.dim() != 2:
            raise ValueError(f"x must be a matrix, got {tuple(x.shape)}")
        tokens, D, F = x.shape[0], self.width, self.hidden
        m = self._matrix
        lddy, ldx = m("dy", dy, tokens, D), m("x", x, tokens, D)
        ldg, ldu, ldd = m("w_gate", w_gate, F, D), m("w_up", w_up, F, D), m("w_down", w_down, D, F)
        g, u, h = saved
        for name, t in (("saved g", g), ("saved u", u), ("saved h", h)):
            if m(name, t, tokens, F) != F:
                raise ValueError(f"{name} must be contiguous")
        new = {"dtype": self.torch_dtype, "device": self.device}
        empty = _torch.empty
        dx, dw_gate, dw_up = empty((tokens, D), **new), empty((F, D), **new), empty((F, D), **new)
        dw_down, dg, du = empty((D, F), **new), empty((tokens, F), **new), empty((tokens, F), **new)
        rc = _L.tgemm_ffn_backward(
            self.handle, tokens, dy.data_ptr(), lddy, x.data_ptr(), ldx, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu,
            w_down.data_ptr(), ldd, g.data_ptr(), u.data_ptr(), h.data_ptr(), dx.data_ptr(), D, dw_gate.data_ptr(),
            dw_up.data_ptr(), dw_down.data_ptr(), dg.data_ptr(), du.data_ptr(), _stream_ptr(self.index))
        if rc:
            raise _tg.TgemmError(rc, f"tgemm_ffn_backward(tokens={tokens}, width={D}, hidden={F})")
        return dx, dw_gate, dw_up, dw_down

    def status(self):
        """Read and clear the device status word; (code, detail)."""
        d = (ctypes.c_int * 4)()
        return int(_L.tgemm_ffn_status(self.handle, d)), list(d)

    def set_watchdog_ns(self, ns):
        _L.tgemm_ffn_set_watchdog_ns(self.handle, ns)

    def debug_stall(self, on):
        _L.tgemm_ffn_debug_stall(self.handle, 1 if on else 0)

    def close(self):
        if self.handle is not None:
            _L.tgemm_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# Plans of gated_ffn(), 16 bytes of device memory each, kept for the process.
_ffn_plans = {}
_ffn_lock = threading.Lock()


def _ffn_plan(x, w_gate, activation):
    if _L is None:
        _setup()
    index = _tensor("x", x)
    if x.dim() != 2 or w_gate.dim() != 2:
        raise ValueError(f"x and w_gate must be matrices, got {tuple(x.shape)} and {tuple(w_gate.shape)}")
    key = (x.shape[1], w_gate.shape[0], x.dtype, activation, index)
    plan = _ffn_plans.get(key)
    if plan is None:
        with _ffn_lock:
            plan = _ffn_plans.get(key)
            if plan is None:
                plan = _ffn_plans[key] = GatedFFN(x.shape[1], w_gate.shape[0], _code("x", x), activation)
    return plan


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", save=False, stream=None):
    """``(act(x Wg^T) * (x Wu^T)) Wd^T``; see `GatedFFN`.  With ``save``: ``(y, saved)`` for `gated_ffn_backward`."""
    return _ffn_plan(x, w_gate, activation).forward(x, w_gate, w_up, w_down, save, stream)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, activation="silu", stream=None):
    """``(dx, dw_gate, dw_up, dw_down)`` of `gated_ffn`; see `GatedFFN.backward`."""
    return _ffn_plan(x, w_gate, activation).backward(dy, x, w_gate, w_up, w_down, saved, stream)

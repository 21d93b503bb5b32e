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

_CODES = None  # torch dtype -> dtype code, filled on first use (torch is imported late)


def _codes():
    global _CODES
    if _CODES is None:
        import torch

        _CODES = {torch.float16: _tg.F16, torch.bfloat16: _tg.BF16, torch.float32: _tg.F32}
    return _CODES


def _on_stream(stream, function, *args, **kwargs):
    """function(*args, **kwargs) with `stream` as the current stream."""
    import torch

    with torch.cuda.stream(stream):
        result = function(*args, **kwargs)
    for t in list(args) + list(kwargs.values()):
        for x in t if isinstance(t, (tuple, list)) else (t,):
            if isinstance(x, torch.Tensor) and x.is_cuda:
                x.record_stream(stream)
    return result


def _require(ok, message, error=ValueError):
    if not ok:
        raise error(message)


def _device_index(name, t):
    """The index of the CUDA device `t` lives on, which has to be the current one."""
    import torch

    _require(isinstance(t, torch.Tensor), f"{name} must be a tensor", TypeError)
    _require(t.is_cuda, f"{name} must be a CUDA tensor")
    index = t.get_device()
    _require(index == torch.cuda.current_device(), f"{name} must be on the current CUDA device")
    return index


def _raise(rc, what):
    raise _tg.TgemmError(rc, what)


def _stream_ptr():
    import torch

    return torch.cuda.current_stream().cuda_stream


def _rows(name, t, width):
    """(rows, elements from one row to the next) of a tensor whose last dimension holds rows of `width`."""
    _require(t.dim() >= 1 and t.shape[-1] == width, f"{name} must have a last dimension of {width}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return (t.numel() // width if width else 0), width
    _require(t.dim() == 2 and t.stride(1) == 1, f"{name} must be contiguous, or a matrix with contiguous rows")
    rows, ld = t.shape[0], t.stride(0)
    if rows <= 1:
        return rows, width
    _require(ld >= width, f"the rows of {name} must not overlap")
    return rows, ld


def _weights(name, t, width, x, index):
    import torch

    _require(isinstance(t, torch.Tensor), f"{name} must be a tensor", TypeError)
    _require(t.get_device() == index, f"{name} must be on x's device")
    _require(t.shape == (width,), f"{name} must have shape ({width},), got {tuple(t.shape)}")
    _require(t.is_contiguous(), f"{name} must be contiguous")
    _require(t.dtype == x.dtype or t.dtype == torch.float32, f"{name} must be {x.dtype} or torch.float32, got {t.dtype}",
             TypeError)
    return t.dtype


def layer_norm(x, weight=None, bias=None, eps=1e-5, stats=False, stream=None):
    """``(x - mean) / sqrt(var + eps) * weight + bias`` over the last dimension of x.

    x is fp16, bf16 or fp32: contiguous, or a matrix with contiguous rows.
    weight and bias (or None) share one type, x's or fp32.  With ``stats`` the
    result is ``(y, mean, rstd)``; mean and rstd are fp32, one value a row, as
    `layer_norm_backward` takes them.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, eps, stats)
    import torch

    index = _device_index("x", x)
    code = _codes().get(x.dtype)
    _require(code is not None, f"x must be fp16, bf16 or fp32, got {x.dtype}", TypeError)
    _require(x.dim() >= 1, "x must have at least one dimension")
    width = x.shape[-1]
    _require(width >= 1, "x must have a last dimension of at least 1")
    rows, ld = _rows("x", x, width)
    wcode = code
    if weight is not None:
        wcode = _codes()[_weights("weight", weight, width, x, index)]
    if bias is not None:
        bcode = _codes()[_weights("bias", bias, width, x, index)]
        _require(weight is None or bcode == wcode, "weight and bias must have the same type", TypeError)
        wcode = bcode
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    mean = rstd = None
    if stats:
        mean, rstd = torch.empty((2, rows), dtype=torch.float32, device=x.device).unbind(0)
    rc = _tg.load().tgemm_layer_norm(
        rows, width, code, wcode, x.data_ptr(), ld, weight.data_ptr() if weight is not None else None,
        bias.data_ptr() if bias is not None else None, eps, y.data_ptr(), width, mean.data_ptr() if stats else None,
        rstd.data_ptr() if stats else None, _stream_ptr())
    if rc != _tg.OK:
        _raise(rc, f"layer_norm(rows={rows}, width={width})")
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, mean, rstd, weight=None, stream=None):
    """``(dx, dweight, dbias)`` of `layer_norm` from the gradient dy of its result.

    mean and rstd are what ``layer_norm(..., stats=True)`` returned.  dweight
    and dbias have weight's type, or x's without a weight.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, mean, rstd, weight)
    import torch

    index = _device_index("x", x)
    code = _codes().get(x.dtype)
    _require(code is not None, f"x must be fp16, bf16 or fp32, got {x.dtype}", TypeError)
    _require(x.dim() >= 1, "x must have at least one dimension")
    width = x.shape[-1]
    _require(width >= 1, "x must have a last dimension of at least 1")
    _device_index("dy", dy)
    _require(dy.dtype == x.dtype, f"dy must be {x.dtype}, got {dy.dtype}", TypeError)
    _require(dy.shape == x.shape, f"dy must have shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    rows, ldx = _rows("x", x, width)
    _, lddy = _rows("dy", dy, width)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _device_index(name, t)
        _require(t.dtype == torch.float32, f"{name} must be torch.float32, got {t.dtype}", TypeError)
        _require(t.numel() == rows and t.is_contiguous(), f"{name} must be contiguous with one value a row")
    wdtype = x.dtype if weight is None else _weights("weight", weight, width, x, index)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw, db = torch.empty((2, width), dtype=wdtype, device=x.device).unbind(0)
    L = _tg.load()
    need = L.tgemm_layer_norm_workspace(rows, width)
    if need < 0:
        _raise(-need, f"layer_norm_backward(rows={rows}, width={width})")
    work = torch.empty(need, dtype=torch.uint8, device=x.device)
    rc = L.tgemm_layer_norm_backward(
        rows, width, code, _codes()[wdtype], dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(),
        weight.data_ptr() if weight is not None else None, dx.data_ptr(), width, dw.data_ptr(), db.data_ptr(),
        work.data_ptr(), need, _stream_ptr())
    if rc != _tg.OK:
        _raise(rc, f"layer_norm_backward(rows={rows}, width={width})")
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
    import torch

    _device_index("x", x)
    code = _codes().get(x.dtype)
    _require(code is not None, f"x must be fp16, bf16 or fp32, got {x.dtype}", TypeError)
    _require(x.is_contiguous(), "x must be contiguous")
    _require(0 <= p <= 1, f"p must lie between 0 and 1, got {p}")
    if residual is not None:
        _device_index("residual", residual)
        _require(residual.dtype == x.dtype, f"residual must be {x.dtype}, got {residual.dtype}", TypeError)
        _require(residual.shape == x.shape, f"residual must have shape {tuple(x.shape)}, got {tuple(residual.shape)}")
        _require(residual.is_contiguous(), "residual must be contiguous")
    y = torch.empty_like(x)
    rc = _tg.load().tgemm_dropout(x.numel(), code, x.data_ptr(), residual.data_ptr() if residual is not None else None,
                                  y.data_ptr(), p, seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF,
                                  _stream_ptr())
    if rc != _tg.OK:
        _raise(rc, f"dropout(n={x.numel()}, p={p})")
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
        _require(activation in _ACTIVATIONS, f"activation must be one of {', '.join(_ACTIVATIONS)}, got {activation!r}")
        self.width, self.hidden, self.activation = int(width), int(hidden), activation
        self.dtype = _tg._dt(dtype)
        h = ctypes.c_void_p()
        self.handle = None
        rc = _tg.load().tgemm_ffn_plan(ctypes.byref(h), self.width, self.hidden, self.dtype, _ACTIVATIONS[activation])
        if rc != _tg.OK:
            _raise(rc, f"tgemm_ffn_plan(width={width}, hidden={hidden}, activation={activation})")
        self.handle = h
        self.torch_dtype = _tg._torch_dtype(self.dtype)
        import torch

        self.device = torch.device("cuda", torch.cuda.current_device())

    def _matrix(self, name, t, rows, cols):
        """(pointer, elements from row to row) of a matrix argument."""
        _require(t.dtype == self.torch_dtype, f"{name} must be {self.torch_dtype}, got {t.dtype}", TypeError)
        _require(t.device == self.device, f"{name} must be on {self.device}, got {t.device}")
        _require(t.shape == (rows, cols), f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
        if rows <= 1 or t.is_contiguous():
            _require(rows == 0 or cols == 1 or t.stride(1) == 1, f"the rows of {name} must be contiguous")
            return t.data_ptr(), cols
        _require(t.stride(1) == 1 and t.stride(0) >= cols, f"the rows of {name} must be contiguous and must not overlap")
        return t.data_ptr(), t.stride(0)

    def _weights(self, w_gate, w_up, w_down):
        D, F = self.width, self.hidden
        return (*self._matrix("w_gate", w_gate, F, D), *self._matrix("w_up", w_up, F, D),
                *self._matrix("w_down", w_down, D, F))

    def forward(self, x, w_gate, w_up, w_down, save=False, stream=None):
        """y, or with ``save`` ``(y, (g, u, h))``: what `backward` takes."""
        if stream is not None:
            return _on_stream(stream, self.forward, x, w_gate, w_up, w_down, save)
        import torch

        _require(x.dim() == 2, f"x must be a matrix, got {tuple(x.shape)}")
        tokens, D, F = x.shape[0], self.width, self.hidden
        args = (*self._matrix("x", x, tokens, D), *self._weights(w_gate, w_up, w_down))
        y = torch.empty((tokens, D), dtype=self.torch_dtype, device=self.device)
        g, u, h = (torch.empty((tokens, F), dtype=self.torch_dtype, device=self.device) if save or i == 2 else None
                   for i in range(3))
        rc = _tg.load().tgemm_ffn_forward(self.handle, tokens, *args, y.data_ptr(), D, g.data_ptr() if save else None,
                                          u.data_ptr() if save else None, h.data_ptr(), _stream_ptr())
        if rc != _tg.OK:
            _raise(rc, f"tgemm_ffn_forward(tokens={tokens}, width={D}, hidden={F})")
        return (y, (g, u, h)) if save else y

    def backward(self, dy, x, w_gate, w_up, w_down, saved, stream=None):
        """``(dx, dw_gate, dw_up, dw_down)`` from the gradient dy of y and what ``forward(..., save=True)`` saved."""
        if stream is not None:
            return _on_stream(stream, self.backward, dy, x, w_gate, w_up, w_down, saved)
        import torch

        _require(x.dim() == 2, f"x must be a matrix, got {tuple(x.shape)}")
        tokens, D, F = x.shape[0], self.width, self.hidden
        args = (*self._matrix("dy", dy, tokens, D), *self._matrix("x", x, tokens, D),
                *self._weights(w_gate, w_up, w_down))
        for name, t in zip(("saved g", "saved u", "saved h"), saved):
            _require(self._matrix(name, t, tokens, F)[1] == F, f"{name} must be contiguous")
        new = {"dtype": self.torch_dtype, "device": self.device}
        dx, dw_gate, dw_up = torch.empty((tokens, D), **new), torch.empty((F, D), **new), torch.empty((F, D), **new)
        dw_down, dg, du = torch.empty((D, F), **new), torch.empty((tokens, F), **new), torch.empty((tokens, F), **new)
        rc = _tg.load().tgemm_ffn_backward(
            self.handle, tokens, *args, *(t.data_ptr() for t in saved), dx.data_ptr(), D, dw_gate.data_ptr(),
            dw_up.data_ptr(), dw_down.data_ptr(), dg.data_ptr(), du.data_ptr(), _stream_ptr())
        if rc != _tg.OK:
            _raise(rc, f"tgemm_ffn_backward(tokens={tokens}, width={D}, hidden={F})")
        return dx, dw_gate, dw_up, dw_down

    def status(self):
        """Read and clear the device status word; (code, detail)."""
        d = (ctypes.c_int * 4)()
        return int(_tg.load().tgemm_ffn_status(self.handle, d)), list(d)

    def set_watchdog_ns(self, ns):
        _tg.load().tgemm_ffn_set_watchdog_ns(self.handle, ns)

    def debug_stall(self, on):
        _tg.load().tgemm_ffn_debug_stall(self.handle, 1 if on else 0)

    def close(self):
        if self.handle is not None:
            _tg.load().tgemm_ffn_destroy(self.handle)
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
    _device_index("x", x)
    _require(x.dim() == 2 and w_gate.dim() == 2, "x and w_gate must be matrices")
    key = (x.shape[1], w_gate.shape[0], x.dtype, activation, x.get_device())
    plan = _ffn_plans.get(key)
    if plan is None:
        _require(x.dtype in _codes(), f"x must be fp16 or bf16, got {x.dtype}", TypeError)
        with _ffn_lock:
            plan = _ffn_plans.get(key)
            if plan is None:
                plan = _ffn_plans[key] = GatedFFN(x.shape[1], w_gate.shape[0], _codes()[x.dtype], activation)
    return plan


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", save=False, stream=None):
    """``(act(x Wg^T) * (x Wu^T)) Wd^T``; see `GatedFFN`.  With ``save``: ``(y, saved)`` for `gated_ffn_backward`."""
    return _ffn_plan(x, w_gate, activation).forward(x, w_gate, w_up, w_down, save, stream)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, activation="silu", stream=None):
    """``(dx, dw_gate, dw_up, dw_down)`` of `gated_ffn`; see `GatedFFN.backward`."""
    return _ffn_plan(x, w_gate, activation).backward(dy, x, w_gate, w_up, w_down, saved, stream)

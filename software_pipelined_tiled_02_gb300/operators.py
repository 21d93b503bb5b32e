"""The feed-forward operators on torch tensors: argument checks, outputs and
workspaces around the C ABI's ``tgemm_layer_norm``, ``tgemm_dropout`` and their
backward passes.

Every function enqueues on torch's current stream and returns at once.  With
``stream`` it runs on that stream instead: outputs and workspaces are then
allocated for it, and the inputs are kept from reuse until it has passed the
call; ordering it after the inputs' producers stays with the caller.
"""

from __future__ import annotations

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

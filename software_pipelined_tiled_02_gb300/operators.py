"""The feed-forward operators on torch tensors: ``layer_norm``, ``gated_ffn``
and ``dropout`` with their backward passes, the same block as a mixture of
experts (``route`` and ``expert_ffn`` with theirs), and products with 4-bit
weights (``gemm_w4``).

The argument checks, the allocation of outputs and workspaces and the calls of
the C ABI (``tgemm_layer_norm``, ``tgemm_ffn_*``, ``tgemm_dropout``,
``tgemm_route``, ``tgemm_experts_*``, ``tgemm_gemm_fourbit``) are made by the
extension module built from ``csrc/binding.cpp``.  Wrong types raise TypeError,
other arguments that do not fit ValueError, and what the library refuses
TgemmError.

Every function enqueues on torch's current stream and returns at once.  With
``stream`` it runs on that stream instead: outputs and workspaces are then
allocated for it, and the inputs are kept from reuse until it has passed the
call; ordering it after the inputs' producers stays with the caller.

None of the functions takes part in autograd: their results are detached, also
those of tensors that require gradients.  The backward passes are functions of
their own, to be called by hand or from a ``torch.autograd.Function``, as in
``examples/feed_forward.py`` and ``examples/mixture_of_experts.py``.
"""

from __future__ import annotations

import ctypes
import operator
import threading

import software_pipelined_tiled_02_gb300 as _tg

_binding = None  # the extension module, bound to the loaded library on first use (torch is imported late)
_lock = threading.Lock()


def _bind():
    global _binding
    with _lock:
        if _binding is None:
            import torch  # noqa: F401  (the extension module needs its libraries)

            L = _tg.load()
            try:
                from . import _binding as module
            except ImportError as e:
                raise RuntimeError(f"_binding.so is missing or does not load ({e}); run "
                                   "software_pipelined_tiled_02_gb300/build.py or __graft_entry__.build()") from e
            functions = (L.tgemm_layer_norm, L.tgemm_layer_norm_workspace, L.tgemm_layer_norm_backward, L.tgemm_dropout,
                         L.tgemm_ffn_forward, L.tgemm_ffn_backward, L.tgemm_route, L.tgemm_route_backward, L.tgemm_gemm_fourbit,
                         L.tgemm_experts_workspace, L.tgemm_experts_forward, L.tgemm_experts_backward)
            module.bind(tuple(ctypes.cast(f, ctypes.c_void_p).value for f in functions), _tg.TgemmError)
            _binding = module
    return _binding


def _on_stream(stream, function, *args):
    """function(*args) with `stream` as the current stream."""
    import torch

    with torch.cuda.stream(stream):
        result = function(*args)
    for a in args:
        for t in a if isinstance(a, tuple) else (a,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return result


def layer_norm(x, weight=None, bias=None, eps=1e-5, stats=False, stream=None):
    """``(x - mean) / sqrt(var + eps) * weight + bias`` over the last dimension of x.

    x is fp16, bf16 or fp32: contiguous, or a matrix with contiguous rows.
    weight and bias (or None) share one type, x's or fp32.  With ``stats`` the
    result is ``(y, mean, rstd)``; mean and rstd are fp32, one value a row, as
    `layer_norm_backward` takes them.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, eps, stats)
    return (_binding or _bind()).layer_norm(x, weight, bias, eps, stats)


def layer_norm_backward(dy, x, mean, rstd, weight=None, stream=None):
    """``(dx, dweight, dbias)`` of `layer_norm` from the gradient dy of its result.

    mean and rstd are what ``layer_norm(..., stats=True)`` returned.  dweight
    and dbias have weight's type, or x's without a weight.
    """
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, mean, rstd, weight)
    return (_binding or _bind()).layer_norm_backward(dy, x, mean, rstd, weight)


def dropout(x, p, seed, offset=0, residual=None, stream=None):
    """x with each element dropped with probability p, the others over 1 - p, plus residual.

    The mask is a function of (seed, offset) and the element's place alone
    (Philox4x32-10; include/tgemm.h has the layout), so `dropout_backward` with
    the same numbers meets the same mask.  seed and offset are taken modulo
    2^64; calls that share a seed take different offsets.
    """
    if stream is not None:
        return _on_stream(stream, dropout, x, p, seed, offset, residual)
    return (_binding or _bind()).dropout(x, p, seed, offset, residual)


def dropout_backward(dy, p, seed, offset=0, stream=None):
    """The gradient of `dropout`'s x (that of its residual is dy itself)."""
    if stream is not None:
        return _on_stream(stream, dropout, dy, p, seed, offset)
    return (_binding or _bind()).dropout(dy, p, seed, offset, None)


_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


class GatedFFN:
    """A plan of the gated feed-forward block ``y = (act(x Wg^T) * (x Wu^T)) Wd^T`` on the current device.

    x is a matrix [tokens, width] with any number of tokens, w_gate and w_up
    are [hidden, width], w_down is [width, hidden]; all fp16 or all bf16, rows
    contiguous and on 16-byte boundaries, width and hidden multiples of 8.
    activation: "silu", "gelu" (the exact one) or "relu".  A plan may be used
    from several threads and on several streams.
    """

    def __init__(self, width, hidden, dtype="bf16", activation="silu"):
        self.handle = None
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}, got {activation!r}")
        self._b = _binding or _bind()
        self.width, self.hidden, self.activation = operator.index(width), operator.index(hidden), activation
        try:
            self.dtype = _tg._dt(dtype)
        except KeyError:
            raise TypeError(f"dtype must be fp16 or bf16, got {dtype!r}") from None
        h = ctypes.c_void_p()
        rc = _tg.load().tgemm_ffn_plan(ctypes.byref(h), self.width, self.hidden, self.dtype, _ACTIVATIONS[activation])
        if rc != _tg.OK:
            raise _tg.TgemmError(rc, f"tgemm_ffn_plan(width={width}, hidden={hidden}, activation={activation})")
        import torch

        self.handle = h
        self._plan = (h.value, self.width, self.hidden, self.dtype, torch.cuda.current_device())

    def forward(self, x, w_gate, w_up, w_down, save=False, stream=None):
        """y, or with ``save`` ``(y, (g, u, h))``: what `backward` takes."""
        if stream is not None:
            return _on_stream(stream, self.forward, x, w_gate, w_up, w_down, save)
        return self._b.ffn_forward(self._plan, x, w_gate, w_up, w_down, save)

    def backward(self, dy, x, w_gate, w_up, w_down, saved, stream=None):
        """``(dx, dw_gate, dw_up, dw_down)`` from the gradient dy of y and what ``forward(..., save=True)`` saved."""
        if stream is not None:
            return _on_stream(stream, self.backward, dy, x, w_gate, w_up, w_down, saved)
        return self._b.ffn_backward(self._plan, dy, x, w_gate, w_up, w_down, saved)

    def kernels(self, tokens):
        """{product: (kernel, CTAs of a cluster)} of a forward and a backward pass over `tokens` tokens: products "up"
        (g, u, h), "down" (y), "dh" (dg, du), "dx" and "dw" (the weight gradients); kernels "pairs", "few" and "rows"."""
        info = (ctypes.c_int * 10)()
        rc = _tg.load().tgemm_ffn_get_kernels(self.handle, operator.index(tokens), info)
        if rc != _tg.OK:
            raise _tg.TgemmError(rc, f"tgemm_ffn_get_kernels({tokens})")
        return {name: (("pairs", "few", "rows")[info[2 * i]], info[2 * i + 1])
                for i, name in enumerate(("up", "down", "dh", "dx", "dw"))}

    def status(self):
        """Read and clear the device status word; (code, detail)."""
        d = (ctypes.c_int * 4)()
        return int(_tg.load().tgemm_ffn_status(self.handle, d)), list(d)

    def set_watchdog_ns(self, ns):
        _tg.load().tgemm_ffn_set_watchdog_ns(self.handle, ns)

    def debug_stall(self, on):
        _tg.load().tgemm_ffn_debug_stall(self.handle, 1 if on else 0)

    def close(self):
        """Free the plan; neither it nor a CUDA graph that captured its calls may be used afterwards."""
        if self.handle is not None:
            self._plan = None  # a later call raises instead of reaching freed memory
            _tg.load().tgemm_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# Plans of gated_ffn(), kept for the process.
_ffn_plans = {}


def _ffn_plan(x, w_gate, activation):
    try:
        return _ffn_plans[x.size(1), w_gate.size(0), x.dtype, activation, x.get_device()]
    except (KeyError, AttributeError, IndexError):
        pass
    return _new_ffn_plan(x, w_gate, activation)


def _new_ffn_plan(x, w_gate, activation):
    import torch

    for name, t in (("x", x), ("w_gate", w_gate)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
        if t.dim() != 2:
            raise ValueError(f"{name} must be a matrix, got {tuple(t.shape)}")
    if not x.is_cuda or x.get_device() != torch.cuda.current_device():
        raise ValueError(f"x must be on the current CUDA device, got {x.device}")
    key = (x.size(1), w_gate.size(0), x.dtype, activation, x.get_device())
    return _ffn_plans.setdefault(key, GatedFFN(x.size(1), w_gate.size(0), x.dtype, activation))


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", save=False, stream=None):
    """``(act(x Wg^T) * (x Wu^T)) Wd^T``; see `GatedFFN`.  With ``save``: ``(y, saved)`` for `gated_ffn_backward`.

    The plan of each pair of sizes, type, activation and device is made on the
    first call and kept for the process (16 bytes of device memory);
    `gated_ffn_status` tells of kernels that gave up.
    """
    return _ffn_plan(x, w_gate, activation).forward(x, w_gate, w_up, w_down, save, stream)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, activation="silu", stream=None):
    """``(dx, dw_gate, dw_up, dw_down)`` of `gated_ffn`; see `GatedFFN.backward`."""
    return _ffn_plan(x, w_gate, activation).backward(dy, x, w_gate, w_up, w_down, saved, stream)


def gated_ffn_status():
    """Read and clear the status words of the plans behind `gated_ffn` and `gated_ffn_backward`; (code, detail).

    OK, or the code of a plan that has another one, as `GatedFFN.status` returns
    it: ERR_TIMEOUT if a bounded wait of one of its kernels ran out, so that
    outputs of calls since the last reading may be incomplete.  Call it after
    synchronising the streams that ran the calls.
    """
    found = (_tg.OK, [0] * 4)
    for plan in list(_ffn_plans.values()):
        status = plan.status()
        if found[0] == _tg.OK:
            found = status
    return found


def _expert_plan(x, w_gate, activation):
    try:
        return _ffn_plans[x.size(1), w_gate.size(1), x.dtype, activation, x.get_device()]
    except (KeyError, AttributeError, IndexError):
        pass
    import torch

    if isinstance(w_gate, torch.Tensor):
        if w_gate.dim() != 3 or w_gate.size(0) < 1:
            raise ValueError(f"w_gate must be [experts, hidden, width], got {tuple(w_gate.shape)}")
        w_gate = w_gate[0]
    return _new_ffn_plan(x, w_gate, activation)


def expert_ffn(x, experts, weights, w_gate, w_up, w_down, activation="silu", save=False, stream=None):
    """Each token's weighted sum of its experts' gated feed-forward blocks.

    x: [tokens, width]; experts and weights: int32 and fp32 [tokens, top],
    contiguous, as `route` returns them (an index out of range takes no part); w_gate and w_up:
    [experts, hidden, width], w_down: [experts, width, hidden]; types, sizes and
    activations as `GatedFFN`'s.  With ``save`` the result is ``(y, saved)``,
    saved = (g, u, h) being what `expert_ffn_backward` takes: [tokens * top,
    hidden], a row for each pair of a token and an existing expert, by expert and
    then by pair; rows behind the last one are undefined.

    Plans are `gated_ffn`'s, and `gated_ffn_status` covers them.
    """
    plan = _expert_plan(x, w_gate, activation)
    if stream is not None:
        return _on_stream(stream, plan._b.experts_forward, plan._plan, x, experts, weights, w_gate, w_up, w_down, save)
    return plan._b.experts_forward(plan._plan, x, experts, weights, w_gate, w_up, w_down, save)


def expert_ffn_backward(dy, x, experts, weights, w_gate, w_up, w_down, saved, activation="silu", stream=None):
    """``(dx, dweights, dw_gate, dw_up, dw_down)`` of `expert_ffn` from the gradient dy of y and what it saved.

    dweights is fp32 [tokens, top], the others have x's type.
    """
    plan = _expert_plan(x, w_gate, activation)
    args = (plan._plan, dy, x, experts, weights, w_gate, w_up, w_down, saved)
    if stream is not None:
        return _on_stream(stream, plan._b.experts_backward, *args)
    return plan._b.experts_backward(*args)


def route(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=None, group_scores=1, renormalize=True,
          scale=1.0, stream=None):
    """Choose top_k experts for each token: ``(weights, experts)``, fp32 and int32, both [tokens, top_k].

    logits: [tokens, experts] fp16, bf16 or fp32 with contiguous rows, up to
    1024 experts.  The scores s are ``softmax(logits)`` or ``sigmoid(logits)``;
    the experts with the largest ``s + bias`` are taken, largest first, ties to
    the lowest index, in the order of exact scores (64 bits of them).  bias (fp32, [experts])
    enters the choice alone; +inf forces an expert, -inf leaves it for last.  With top_groups < groups only experts of the
    top_groups best groups of neighbours can be chosen, by the sum of the
    group's ``group_scores`` (1 or 2) largest keys.  weights are ``scale * s``,
    with ``renormalize`` over the sum of the token's chosen s.  NaN counts as
    larger than all else; where every chosen score is 0 so are the weights.
    """
    if stream is not None:
        return _on_stream(stream, route, logits, top_k, scoring, bias, groups, top_groups, group_scores, renormalize, scale)
    return (_binding or _bind()).route(logits, top_k, scoring, bias, groups, top_groups, group_scores, renormalize, scale)


def route_backward(dweights, logits, experts, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """The gradient of `route`'s logits from that of its weights, for the experts it chose.

    The choice has no gradient, so bias and groups have no part in it.  An
    index out of range counts as not chosen.
    """
    if stream is not None:
        return _on_stream(stream, route_backward, dweights, logits, experts, scoring, renormalize, scale)
    return (_binding or _bind()).route_backward(dweights, logits, experts, scoring, renormalize, scale)


def _dtype_code(dtype):
    try:
        return _tg._dt(dtype)
    except KeyError:  # none of the library's types
        return None


def gemm_w4(x, packed, scales, zeros=None, experts=None, out_dtype=None, stream=None):
    """``x W^T`` for a few rows x and 4-bit weights ``W = (q - zeros) * scales``.

    packed: uint8 [rows, width / 2], weight i of a row in the low (even i) or
    high half of byte i / 2.  scales: [rows, width / group], x's type or fp32;
    group is a multiple of 32.  zeros: uint8 of scales' shape, 0 .. 15, or None:
    8 everywhere.  x: fp16 or bf16, [..., width]; the result [..., rows] has x's
    type or fp32 (``out_dtype``).

    With ``experts`` (int32 [tokens, top]) packed, scales and zeros are stacks of
    matrices, [experts, ...], x is [tokens, width] or [tokens, top, width], and
    the result [tokens, top, rows] takes for each pair the matrix that its index
    names; rows of an index out of range are 0.

    The weights are read once for every 32 rows, with ``experts`` for every 8,
    16 or 32 of a matrix's pairs, by how many it has on average.  A row's last
    bits may depend on the number of rows.
    """
    if stream is not None:
        return _on_stream(stream, gemm_w4, x, packed, scales, zeros, experts, out_dtype)
    f32 = False
    if out_dtype is not None:
        code, own = _dtype_code(out_dtype), _dtype_code(getattr(x, "dtype", None))
        f32 = code == _tg.F32
        if not f32 and own is not None and code != own:
            raise TypeError(f"out_dtype must be x's type or fp32, got {out_dtype!r}")
    return (_binding or _bind()).gemm_w4(x, packed, scales, zeros, experts, f32)

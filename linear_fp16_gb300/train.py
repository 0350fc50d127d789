"""The two ends of a training step: ctypes binding and tensor-level calls.

``linear_cross_entropy`` is the softmax cross entropy of a vocabulary head z =
x W^T + b, without the logits in memory, and ``linear_cross_entropy_backward``
its gradients.  ``adamw_step`` updates a list of parameters with the clipped
gradients; ``adamw_state`` makes the state that it keeps, in 32 or in 8 bits.  Like the feed-forward calls
(``ffn``) they record no graph for torch's automatic differentiation: tensors
that require gradients are taken as values.  The functions named like the C
entry points (include/poot_train.h) take the argument structures and return
the status code; every step of the computation runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
import threading

from . import binding as _b
from . import ffn as _ffn

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class LinearCrossEntropyArgs(ctypes.Structure):
    """struct poot_linear_cross_entropy_args."""
    _fields_ = ([(n, _VP) for n in ("x", "w", "b", "target", "loss", "lse")]
                + [(n, _I64) for n in ("M", "V", "K", "ldx", "ignore_index")] + [("dtype", _INT)])


class LinearCrossEntropyBackwardArgs(ctypes.Structure):
    """struct poot_linear_cross_entropy_backward_args."""
    _fields_ = ([(n, _VP) for n in ("dloss", "x", "w", "b", "target", "lse", "dx", "dw", "db")]
                + [(n, _I64) for n in ("M", "V", "K", "ldx", "dloss_stride", "ignore_index")] + [("dtype", _INT)])


class AdamwTensor(ctypes.Structure):
    """struct poot_adamw_tensor."""
    _fields_ = ([(n, _VP) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "copy")]
                + [("n", _I64), ("weight_decay", ctypes.c_double)]
                + [(n, _INT) for n in ("param_dtype", "grad_dtype", "copy_dtype")])


class AdamwArgs(ctypes.Structure):
    """struct poot_adamw_args."""
    _fields_ = ([("tensors", ctypes.POINTER(AdamwTensor)), ("count", _I64)]
                + [(n, _VP) for n in ("lr_device", "step_device", "grad_scale_device")] + [("step", _I64)]
                + [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "grad_scale")] + [("bits", _INT)])


class AdamwCodes(ctypes.Structure):
    """struct poot_adamw_codes."""
    _fields_ = [(n, _VP) for n in ("m", "v", "m_scale", "v_scale", "m_out", "v_out")] + [("n", _I64)]


# (restype, argtypes) of every function of include/poot_train.h
EXPORTS = {
    "poot_linear_cross_entropy": (_INT, [ctypes.POINTER(LinearCrossEntropyArgs), _VP]),
    "poot_linear_cross_entropy_backward": (_INT, [ctypes.POINTER(LinearCrossEntropyBackwardArgs), _VP]),
    "poot_adamw_step": (_INT, [ctypes.POINTER(AdamwArgs), _VP]),
    "poot_adamw_values": (_INT, [ctypes.POINTER(AdamwCodes), _I64, _VP]),
}

_lock = threading.Lock()
_lib = None


def load_library() -> ctypes.CDLL:
    """The CUDA library with the functions of include/poot_train.h bound."""
    global _lib
    if _lib is None:
        lib = _b.load_library()
        with _lock:
            for name, (res, args) in EXPORTS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


# ---- raw C entry points --------------------------------------------------
def _ref(args):
    return ctypes.byref(args) if args is not None else None


def poot_linear_cross_entropy(args, stream: int) -> int:
    """args: a LinearCrossEntropyArgs instance."""
    return load_library().poot_linear_cross_entropy(_ref(args), stream)


def poot_linear_cross_entropy_backward(args, stream: int) -> int:
    """args: a LinearCrossEntropyBackwardArgs instance."""
    return load_library().poot_linear_cross_entropy_backward(_ref(args), stream)


def poot_adamw_step(args, stream: int) -> int:
    """args: an AdamwArgs instance."""
    return load_library().poot_adamw_step(_ref(args), stream)


def poot_adamw_values(states, count: int, stream: int) -> int:
    """states: an array of AdamwCodes (or None with count 0)."""
    return load_library().poot_adamw_values(states, count, stream)


# ---- tensor-level calls (checks and allocation: csrc/train_calls.h) ----------
def _calls():
    return _ffn._ext or _ffn.load_tensor_calls()


def linear_cross_entropy(x, w, target, bias=None, *, ignore_index: int = -100, save: bool = False, stream=None):
    """loss[i] = log sum_v exp z[i, v] - z[i, target[i]] for z = x W^T + bias.

    x [M,K] (unit column stride, rows may be further apart), w [V,K]
    contiguous, bias [V] or None: float16 or bfloat16 CUDA tensors of one
    dtype; target [M] int64.  Returns the rows' losses, float32 [M]: 0 where
    the target is ``ignore_index``, NaN where it is outside [0, V) otherwise.  With ``save``
    returns (loss, lse): the rows' log-sum-exp, which
    linear_cross_entropy_backward reads.  The logits are never in memory.
    Streams and errors as in gated_linear.
    """
    r = _calls().linear_cross_entropy(x, w, target, bias, ignore_index, save, _ffn._stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_linear_cross_entropy")
    return r


def linear_cross_entropy_backward(dloss, x, w, target, lse, bias=None, *, ignore_index: int = -100,
                                  need_dx: bool = True, need_dw: bool = True, need_db: bool = False, stream=None):
    """Gradients (dx, dw, db) of sum(dloss * loss); None where not needed.

    dloss: float32 [M], any stride of 0 or more: a mean over n rows is
    ``torch.full((1,), 1 / n, device=...).expand(M)``.  lse is what
    linear_cross_entropy returned with ``save``; the logits are computed again,
    a piece of the vocabulary at a time.  Rows under ``ignore_index`` contribute
    nothing, whatever they hold; their dx is 0.  In float16 the loss scale of
    a training step belongs into dloss.
    """
    r = _calls().linear_cross_entropy_backward(dloss, x, w, target, lse, bias, ignore_index, need_dx, need_dw, need_db,
                                               _ffn._stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_linear_cross_entropy_backward")
    return r


ADAMW_BLOCK = 256  # elements that share a scale of an 8-bit state


class AdamWState:
    """The averages m and v that adamw_step keeps for a list of parameters.

    32 bits: lists ``m`` and ``v`` of float32 tensors, shaped like the
    parameters.  8 bits: int8 ``m`` and uint8 ``v``, shaped likewise, with float32
    ``m_scale`` and ``v_scale`` of one element for each 256 of a parameter, in order
    (include/poot_train.h has the codes).  The lists may be saved and
    given again; ``adamw_state`` makes them for a first step.
    """

    def __init__(self, m, v, m_scale=None, v_scale=None):
        self.m, self.v = list(m), list(v)
        self.m_scale, self.v_scale = list(m_scale or ()) or None, list(v_scale or ()) or None

    @property
    def bits(self) -> int:
        return 32 if self.m_scale is None else 8

    def values(self, *, stream=None):
        """(m, v): lists of float32 tensors; with 8 bits new ones, what the codes stand for."""
        if self.m_scale is None:
            return self.m, self.v
        r = _calls().adamw_values(self.m, self.v, self.m_scale, self.v_scale, _ffn._stream(stream))
        if r.__class__ is int:
            raise _b.PootLinearError(r, "poot_adamw_values")
        return r


def adamw_state(params, *, bits: int = 32) -> AdamWState:
    """A state of zeros for adamw_step, beside each of the parameters."""
    import torch
    if bits not in (32, 8):
        raise ValueError(f"bits must be 32 or 8, not {bits!r}")
    params = list(params)

    def zeros(dtype, shape=None):
        return [torch.zeros(p.shape if shape is None else shape(p), dtype=dtype, device=p.device) for p in params]
    if bits == 32:
        return AdamWState(zeros(torch.float32), zeros(torch.float32))

    def blocks(p):
        return -(-p.numel() // ADAMW_BLOCK)
    return AdamWState(zeros(torch.int8), zeros(torch.uint8), zeros(torch.float32, blocks), zeros(torch.float32, blocks))


def adamw_step(params, grads, state: AdamWState, *, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay=0.01, grad_scale=1.0, copies=None, stream=None) -> None:
    """One AdamW step over all parameters at once, in place.

    With g = grad * grad_scale: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
    p = p (1 - lr weight_decay) - lr / (1 - b1^step) m / (sqrt(v) / sqrt(1 -
    b2^step) + eps).  params and grads: sequences of contiguous CUDA tensors of
    one device (float16, bfloat16 or float32, any mixture).  ``copies``: a
    sequence of float16 or bfloat16 tensors (or None in places) that receive the
    new values of float32 parameters.  ``weight_decay``: one number, or one for each
    tensor.  ``step`` counts from 1.  ``step`` (int64), ``lr`` and
    ``grad_scale`` (float32) may be CUDA tensors of one element, read when the step
    runs: a captured graph follows them.  Tensors written to count as modified
    in place; ones that require gradients are written all the same.  An empty
    sequence raises ValueError.  Streams and errors as in gated_linear.
    """
    decay = weight_decay if isinstance(weight_decay, (int, float)) else list(weight_decay)
    r = _calls().adamw_step(list(params), list(grads), state.m, state.v, state.m_scale, state.v_scale,
                            None if copies is None else list(copies), decay, step, lr, grad_scale, betas[0], betas[1],
                            eps, _ffn._stream(stream))
    if r is not None:
        raise _b.PootLinearError(r, "poot_adamw_step")

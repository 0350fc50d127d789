"""The two ends of a training step: ctypes binding and tensor-level calls.

``linear_cross_entropy`` is the softmax cross entropy of a vocabulary head z =
x W^T + b, without the logits in memory, and ``linear_cross_entropy_backward``
its gradients.  Like the feed-forward calls
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


# (restype, argtypes) of every function of include/poot_train.h
EXPORTS = {
    "poot_linear_cross_entropy": (_INT, [ctypes.POINTER(LinearCrossEntropyArgs), _VP]),
    "poot_linear_cross_entropy_backward": (_INT, [ctypes.POINTER(LinearCrossEntropyBackwardArgs), _VP]),
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

"""The feed-forward operators: ctypes binding and tensor-level calls.

``gated_linear`` (h = act(x Wg^T + bg) * (x Wu^T + bu)) and its gradients
``gated_linear_backward``, the linear's gradients ``linear_backward``, and
``clip_grad_norm`` over a list of gradients.  The calls record no graph for
torch's automatic differentiation: tensors that require gradients are taken as
values, and the gradients are the calls for them.  The functions named like the C
entry points (include/poot_ffn.h) take the argument structures and return
the status code; every step of the computation runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import threading

from . import binding as _b
from . import build as _build

ACT_SILU = 0
ACT_GELU_TANH = 1
ACT_GELU_ERF = 2
ACT_CODES = {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH, "gelu_erf": ACT_GELU_ERF}
GRAD_F16 = 0
GRAD_BF16 = 1
GRAD_F32 = 2

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class GatedLinearArgs(ctypes.Structure):
    """struct poot_gated_linear_args."""
    _fields_ = ([(n, _VP) for n in ("x", "wg", "wu", "bg", "bu", "h", "g", "u")]
                + [(n, _I64) for n in ("M", "N", "K", "ldx")] + [("dtype", _INT), ("activation", _INT)])


class GatedLinearBackwardArgs(ctypes.Structure):
    """struct poot_gated_linear_backward_args."""
    _fields_ = ([(n, _VP) for n in ("dh", "x", "wg", "wu", "g", "u", "dx", "dwg", "dwu", "dbg", "dbu")]
                + [(n, _I64) for n in ("M", "N", "K", "ld_dh", "ldx", "ld_g", "ld_u")]
                + [("dtype", _INT), ("activation", _INT)])


class LinearBackwardArgs(ctypes.Structure):
    """struct poot_linear_backward_args."""
    _fields_ = ([(n, _VP) for n in ("dy", "x", "w", "dx", "dw", "db")]
                + [(n, _I64) for n in ("M", "N", "K", "ld_dy", "ldx")] + [("dtype", _INT)])


class GradTensor(ctypes.Structure):
    """struct poot_grad_tensor."""
    _fields_ = [("src", _VP), ("dst", _VP), ("n", _I64), ("dtype", _INT)]


# (restype, argtypes) of every function of include/poot_ffn.h
EXPORTS = {
    "poot_gated_linear": (_INT, [ctypes.POINTER(GatedLinearArgs), _VP]),
    "poot_gated_linear_backward": (_INT, [ctypes.POINTER(GatedLinearBackwardArgs), _VP]),
    "poot_linear_backward": (_INT, [ctypes.POINTER(LinearBackwardArgs), _VP]),
    "poot_clip_grad_norm": (_INT, [ctypes.POINTER(GradTensor), _I64, ctypes.c_float, _VP, _VP]),
}

_lock = threading.Lock()
_lib = None


def load_library() -> ctypes.CDLL:
    """The CUDA library with the functions of include/poot_ffn.h bound."""
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


def poot_gated_linear(args, stream: int) -> int:
    """args: a GatedLinearArgs instance."""
    return load_library().poot_gated_linear(_ref(args), stream)


def poot_gated_linear_backward(args, stream: int) -> int:
    """args: a GatedLinearBackwardArgs instance."""
    return load_library().poot_gated_linear_backward(_ref(args), stream)


def poot_linear_backward(args, stream: int) -> int:
    """args: a LinearBackwardArgs instance."""
    return load_library().poot_linear_backward(_ref(args), stream)


def poot_clip_grad_norm(tensors, count: int, max_norm: float, norm: int, stream: int) -> int:
    """tensors: an array of GradTensor (or None with count 0); norm: device pointer to one float."""
    return load_library().poot_clip_grad_norm(tensors, count, max_norm, norm, stream)


# ---- tensor-level calls ----------------------------------------------------
# The checks of the tensors, the allocation of results and the call of the C
# entry point are in csrc/ffn_torch.cpp: at decode sizes they would take longer
# in Python than the kernels.
_ext = None


def load_tensor_calls():
    """The extension behind the tensor-level calls (built first if needed).

    The C entry points above need the library alone, neither this nor torch.
    """
    global _ext
    if _ext is None:
        path = _build.build_extension()
        load_library()  # comes first: the extension links to it
        loader = importlib.machinery.ExtensionFileLoader("_ffn_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ffn_torch", loader))
        loader.exec_module(module)
        _ext = module
    return _ext


def _act(activation):
    act = ACT_CODES.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}; one of {sorted(ACT_CODES)}")
    return act


def _stream(stream):
    return None if stream is None else (stream.stream_id, stream.device_index, stream.device_type)


def gated_linear(x, wg, wu, bg=None, bu=None, *, activation: str = "silu", save: bool = False, out=None,
                 stream=None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu) in one pass.

    x [M,K] (unit column stride, rows may be further apart), wg and wu [N,K]
    contiguous, bg and bu [N] or None: float16 or bfloat16 CUDA tensors of one
    dtype.  ``activation``: "silu", "gelu_tanh" or "gelu_erf".  Returns h
    [M,N] (``out`` if given), or with ``save`` (h, g, u): the two
    pre-activations, rounded to the dtype, that gated_linear_backward reads.
    No result is attached to torch's autograd graph.
    Runs on ``stream`` (default: the current stream of x's device), which the
    caller orders after the work that makes the inputs; memory of the tensors
    given is not reused before that stream is done with it.  Raises
    PootLinearError on a status other than POOT_OK.
    """
    r = (_ext or load_tensor_calls()).gated_linear(x, wg, wu, bg, bu, out, _act(activation), save, _stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_gated_linear")
    return r


def gated_linear_backward(dh, x, wg, wu, g, u, *, activation: str = "silu", need_dx: bool = True,
                          need_dw: bool = True, need_db: bool = False, stream=None):
    """Gradients (dx, dwg, dwu, dbg, dbu) of gated_linear; None where not needed.

    dh, g and u [M,N] and x [M,K] may have rows further apart than their
    columns; g and u are what gated_linear returned with ``save``.
    """
    r = (_ext or load_tensor_calls()).gated_linear_backward(dh, x, wg, wu, g, u, _act(activation), need_dx, need_dw,
                                                        need_db, _stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_gated_linear_backward")
    return r


def linear_backward(dy, x, w, *, need_dx: bool = True, need_dw: bool = True, need_db: bool = True, stream=None):
    """Gradients (dx, dw, db) of y = x W^T + b for dy [M,N]; None where not needed."""
    r = (_ext or load_tensor_calls()).linear_backward(dy, x, w, need_dx, need_dw, need_db, _stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_linear_backward")
    return r


def clip_grad_norm(grads, max_norm: float, *, out=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm.

    grads: a sequence of contiguous CUDA tensors of one device (float16,
    bfloat16 or float32, any mixture), clipped in place; with ``out``, a
    sequence of tensors of the same shapes and dtypes, the results go there
    instead.  The norm, over all tensors together, is a float32 scalar tensor
    on the device (the call does not synchronise).  Tensors written to count as
    modified in place (their version goes up); ones that require gradients are
    written all the same.  An empty sequence raises ValueError: there is no device
    to put a norm on.
    """
    r = (_ext or load_tensor_calls()).clip_grad_norm(list(grads), None if out is None else list(out), max_norm,
                                                 _stream(stream))
    if r.__class__ is int:
        raise _b.PootLinearError(r, "poot_clip_grad_norm")
    return r

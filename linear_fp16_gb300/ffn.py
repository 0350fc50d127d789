"""The feed-forward operators: ctypes binding and tensor-level calls.

``gated_linear`` (h = act(x Wg^T + bg) * (x Wu^T + bu)) and its gradients
``gated_linear_backward``, the linear's gradients ``linear_backward``, and
``clip_grad_norm`` over a list of gradients.  The functions named like the C
entry points (include/poot_ffn.h) take the argument structures and return
the status code; every step of the computation runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
import threading

from . import binding as _b

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
def _matrix(t, name, shape, like=None):
    """t as a 2-D CUDA tensor of `shape` (None: any extent), unit column stride."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float16, torch.bfloat16) or (like is not None and t.dtype != like.dtype):
        raise TypeError(f"{name} must be float16 or bfloat16, one dtype for all tensors, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if t.dim() != len(shape) or any(w is not None and s != w for s, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


def _rows(t, name, shape, like=None):
    """A matrix whose rows may be further apart than its columns (a view)."""
    _matrix(t, name, shape, like)
    rows, cols = t.shape
    if t.numel() > 0 and ((cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols)):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return t


def _dense(t, name, shape, like=None):
    _matrix(t, name, shape, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _act(activation):
    if activation not in ACT_CODES:
        raise ValueError(f"unknown activation {activation!r}; one of {sorted(ACT_CODES)}")
    return ACT_CODES[activation]


def _dtype(t):
    import torch
    return _b.DTYPE_BF16 if t.dtype == torch.bfloat16 else _b.DTYPE_F16


class _Launch:
    """The stream of a call, and the tensors it allocates: from that stream's
    memory, and kept from reuse while the caller's stream may still read them."""

    def __init__(self, device, stream):
        import torch
        self.current = torch.cuda.current_stream(device)
        self.stream = self.current if stream is None else stream
        self.device = device

    def empty(self, shape, dtype):
        import torch
        if self.stream == self.current:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(self.current)
        return t

    def call(self, fn, name, *args):
        import torch
        with torch.cuda.device(self.device):
            rc = fn(*args, self.stream.cuda_stream)
        if rc != _b.POOT_OK:
            raise _b.PootLinearError(rc, name)


def gated_linear(x, wg, wu, bg=None, bu=None, *, activation: str = "silu", save: bool = False, out=None,
                 stream=None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu) in one pass.

    x [M,K] (unit column stride, rows may be further apart), wg and wu [N,K]
    contiguous, bg and bu [N] or None: float16 or bfloat16 CUDA tensors of one
    dtype.  ``activation``: "silu", "gelu_tanh" or "gelu_erf".  Returns h
    [M,N] (``out`` if given), or with ``save`` (h, g, u): the two
    pre-activations, rounded to the dtype, that gated_linear_backward reads.
    Runs on ``stream`` (default: the current stream of x's device).
    """
    _rows(x, "x", (None, None))
    M, K = x.shape
    _dense(wg, "wg", (None, K), x)
    N = wg.shape[0]
    _dense(wu, "wu", (N, K), x)
    for name, b in (("bg", bg), ("bu", bu)):
        if b is not None:
            _dense(b, name, (N,), x)
    act = _act(activation)
    run = _Launch(x.device, stream)
    if out is None:
        out = run.empty((M, N), x.dtype)
    else:
        _dense(out, "out", (M, N), x)
    g = run.empty((M, N), x.dtype) if save else None
    u = run.empty((M, N), x.dtype) if save else None
    args = GatedLinearArgs(_ptr(x), _ptr(wg), _ptr(wu), _ptr(bg), _ptr(bu), _ptr(out), _ptr(g), _ptr(u), M, N, K,
                           _ld(x), _dtype(x), act)
    run.call(poot_gated_linear, "poot_gated_linear", args)
    return (out, g, u) if save else out


def gated_linear_backward(dh, x, wg, wu, g, u, *, activation: str = "silu", need_dx: bool = True,
                          need_dw: bool = True, need_db: bool = False, stream=None):
    """Gradients (dx, dwg, dwu, dbg, dbu) of gated_linear; None where not needed.

    dh, g and u [M,N] and x [M,K] may have rows further apart than their
    columns; g and u are what gated_linear returned with ``save``.
    """
    _rows(x, "x", (None, None))
    M, K = x.shape
    _dense(wg, "wg", (None, K), x)
    N = wg.shape[0]
    _dense(wu, "wu", (N, K), x)
    for name, t in (("dh", dh), ("g", g), ("u", u)):
        _rows(t, name, (M, N), x)
    act = _act(activation)
    run = _Launch(x.device, stream)
    dx = run.empty((M, K), x.dtype) if need_dx else None
    dwg = run.empty((N, K), x.dtype) if need_dw else None
    dwu = run.empty((N, K), x.dtype) if need_dw else None
    dbg = run.empty((N,), x.dtype) if need_db else None
    dbu = run.empty((N,), x.dtype) if need_db else None
    args = GatedLinearBackwardArgs(_ptr(dh), _ptr(x), _ptr(wg), _ptr(wu), _ptr(g), _ptr(u), _ptr(dx), _ptr(dwg),
                                   _ptr(dwu), _ptr(dbg), _ptr(dbu), M, N, K, _ld(dh), _ld(x), _ld(g), _ld(u),
                                   _dtype(x), act)
    run.call(poot_gated_linear_backward, "poot_gated_linear_backward", args)
    return dx, dwg, dwu, dbg, dbu


def linear_backward(dy, x, w, *, need_dx: bool = True, need_dw: bool = True, need_db: bool = True, stream=None):
    """Gradients (dx, dw, db) of y = x W^T + b for dy [M,N]; None where not needed."""
    _rows(x, "x", (None, None))
    M, K = x.shape
    _dense(w, "w", (None, K), x)
    N = w.shape[0]
    _rows(dy, "dy", (M, N), x)
    run = _Launch(x.device, stream)
    dx = run.empty((M, K), x.dtype) if need_dx else None
    dw = run.empty((N, K), x.dtype) if need_dw else None
    db = run.empty((N,), x.dtype) if need_db else None
    args = LinearBackwardArgs(_ptr(dy), _ptr(x), _ptr(w), _ptr(dx), _ptr(dw), _ptr(db), M, N, K, _ld(dy), _ld(x),
                              _dtype(x))
    run.call(poot_linear_backward, "poot_linear_backward", args)
    return dx, dw, db


def clip_grad_norm(grads, max_norm: float, *, out=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm.

    grads: a sequence of contiguous CUDA tensors of one device (float16,
    bfloat16 or float32, any mixture), clipped in place; with ``out``, a
    sequence of tensors of the same shapes and dtypes, the results go there
    instead.  The norm, over all tensors together, is a float32 scalar tensor
    on the device (the call does not synchronise).
    """
    import torch
    codes = {torch.float16: GRAD_F16, torch.bfloat16: GRAD_BF16, torch.float32: GRAD_F32}
    grads = list(grads)
    dsts = grads if out is None else list(out)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    if len(dsts) != len(grads):
        raise ValueError(f"out must hold {len(grads)} tensors, got {len(dsts)}")
    table = (GradTensor * len(grads))()
    device = grads[0].device if isinstance(grads[0], torch.Tensor) else None
    for i, (g, d) in enumerate(zip(grads, dsts)):
        for name, t in (("grads", g), ("out", d)):
            if not isinstance(t, torch.Tensor) or t.dtype not in codes:
                raise TypeError(f"{name}[{i}] must be a float16, bfloat16 or float32 tensor")
            if not t.is_cuda or t.device != device or not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be a contiguous CUDA tensor on the device of the first")
        if d.dtype != g.dtype or d.shape != g.shape:
            raise ValueError(f"out[{i}] must have the shape and dtype of grads[{i}]")
        table[i] = GradTensor(g.data_ptr(), d.data_ptr(), g.numel(), codes[g.dtype])
    run = _Launch(device, stream)
    norm = run.empty((), torch.float32)
    run.call(poot_clip_grad_norm, "poot_clip_grad_norm", table, len(grads), float(max_norm), norm.data_ptr())
    return norm

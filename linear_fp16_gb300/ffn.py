"""The feed-forward operators: ctypes binding and tensor-level calls.

``gated_linear`` (h = act(x Wg^T + bg) * (x Wu^T + bu)) and its gradients
``gated_linear_backward``, the linear's gradients ``linear_backward``, and
``clip_grad_norm`` over a list of gradients.  The functions named like the C
entry points (include/poot_ffn.h) take the argument structures and return
the status code; every step of the computation runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch

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
# Decode-sized calls take a few microseconds on the GPU, so the host's part
# is kept short: one combined check per tensor (the error texts are made only
# when it fails), the argument structures packed as bytes, the stream handle
# read directly.
_PACK_GATED = struct.Struct("@8P4q2i")
_PACK_GATED_BWD = struct.Struct("@11P7q2i")
_PACK_LINEAR_BWD = struct.Struct("@6P5qi4x")
_PACK_GRAD = struct.Struct("@2Pqi4x")
_packed = {}


def _packed_fn(name):
    """The C function `name` taking its arguments as packed bytes."""
    fn = _packed.get(name)
    if fn is None:
        fn = load_library()[name]  # a function object of its own
        fn.restype = _INT
        args = [ctypes.c_char_p, _VP]
        if name == "poot_clip_grad_norm":
            args = [ctypes.c_char_p, _I64, ctypes.c_float, _VP, _VP]
        fn.argtypes = args
        _packed[name] = fn
    return fn


def _refuse(t, name, dtype, device, shape, dense):
    """Raises what _ok found wrong with t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _CODES or t.dtype != dtype:
        raise TypeError(f"{name} must be float16 or bfloat16, one dtype for all tensors, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous" if dense else
                     f"{name} must have unit column stride and rows that do not overlap")


_CODES = {torch.float16: _b.DTYPE_F16, torch.bfloat16: _b.DTYPE_BF16}


def _first(x):
    """dtype, its code, device index, rows, columns and row pitch of x [M,K]."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype = x.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"x must be float16 or bfloat16, got {dtype}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dims, got {tuple(x.shape)}")
    device = x.get_device()
    M, K = x.shape
    return dtype, code, device, M, K, _pitch(x, "x", dtype, device, (M, K))


def _pitch(t, name, dtype, device, shape):
    """Row pitch of a matrix whose rows may be further apart than its columns."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape):
        _refuse(t, name, dtype, device, shape, False)
    if t.is_contiguous():
        return shape[1]
    rows, cols = shape
    s0, s1 = t.stride()
    if (cols > 1 and s1 != 1) or (rows > 1 and s0 < cols):
        _refuse(t, name, dtype, device, shape, False)
    return s0 if rows > 1 else cols


def _dense(t, name, dtype, device, shape):
    """Address of a contiguous tensor."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape
            and t.is_contiguous()):
        _refuse(t, name, dtype, device, shape, True)
    return t.data_ptr()


def _rows_of(w, name):
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if w.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(w.shape)}")
    return w.shape[0]


def _act(activation):
    act = ACT_CODES.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}; one of {sorted(ACT_CODES)}")
    return act


def _stream(device, stream):
    """(handle, other): the stream's handle, and whether it is not the current one."""
    current = torch._C._cuda_getCurrentRawStream(device)
    if stream is None:
        return current, None
    return stream.cuda_stream, (stream if stream.cuda_stream != current else None)


def _empty(like, shape, other, dtype=None):
    """An output of the call: from its stream's memory, and kept from reuse
    while the caller's current stream may still read it."""
    if dtype is None:
        dtype = like.dtype
    if other is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _call(name, device, *args):
    fn = _packed_fn(name)
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != _b.POOT_OK:
        raise _b.PootLinearError(rc, name)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


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
    dtype, code, dev, M, K, ldx = _first(x)
    N = _rows_of(wg, "wg")
    pg, pu = _dense(wg, "wg", dtype, dev, (N, K)), _dense(wu, "wu", dtype, dev, (N, K))
    pbg = 0 if bg is None else _dense(bg, "bg", dtype, dev, (N,))
    pbu = 0 if bu is None else _dense(bu, "bu", dtype, dev, (N,))
    act = _act(activation)
    handle, other = _stream(dev, stream)
    if out is None:
        out = _empty(x, (M, N), other)
        po = out.data_ptr()
    else:
        po = _dense(out, "out", dtype, dev, (M, N))
    g = u = None
    if save:
        g, u = _empty(x, (M, N), other), _empty(x, (M, N), other)
    _call("poot_gated_linear", dev,
          _PACK_GATED.pack(x.data_ptr(), pg, pu, pbg, pbu, po, _ptr(g), _ptr(u), M, N, K, ldx, code, act), handle)
    return (out, g, u) if save else out


def gated_linear_backward(dh, x, wg, wu, g, u, *, activation: str = "silu", need_dx: bool = True,
                          need_dw: bool = True, need_db: bool = False, stream=None):
    """Gradients (dx, dwg, dwu, dbg, dbu) of gated_linear; None where not needed.

    dh, g and u [M,N] and x [M,K] may have rows further apart than their
    columns; g and u are what gated_linear returned with ``save``.
    """
    dtype, code, dev, M, K, ldx = _first(x)
    N = _rows_of(wg, "wg")
    pg, pu = _dense(wg, "wg", dtype, dev, (N, K)), _dense(wu, "wu", dtype, dev, (N, K))
    ld_dh = _pitch(dh, "dh", dtype, dev, (M, N))
    ld_g, ld_u = _pitch(g, "g", dtype, dev, (M, N)), _pitch(u, "u", dtype, dev, (M, N))
    act = _act(activation)
    handle, other = _stream(dev, stream)
    dx = _empty(x, (M, K), other) if need_dx else None
    dwg, dwu = (_empty(x, (N, K), other), _empty(x, (N, K), other)) if need_dw else (None, None)
    dbg, dbu = (_empty(x, (N,), other), _empty(x, (N,), other)) if need_db else (None, None)
    _call("poot_gated_linear_backward", dev,
          _PACK_GATED_BWD.pack(dh.data_ptr(), x.data_ptr(), pg, pu, g.data_ptr(), u.data_ptr(), _ptr(dx), _ptr(dwg),
                               _ptr(dwu), _ptr(dbg), _ptr(dbu), M, N, K, ld_dh, ldx, ld_g, ld_u, code, act), handle)
    return dx, dwg, dwu, dbg, dbu


def linear_backward(dy, x, w, *, need_dx: bool = True, need_dw: bool = True, need_db: bool = True, stream=None):
    """Gradients (dx, dw, db) of y = x W^T + b for dy [M,N]; None where not needed."""
    dtype, code, dev, M, K, ldx = _first(x)
    N = _rows_of(w, "w")
    pw = _dense(w, "w", dtype, dev, (N, K))
    ld_dy = _pitch(dy, "dy", dtype, dev, (M, N))
    handle, other = _stream(dev, stream)
    dx = _empty(x, (M, K), other) if need_dx else None
    dw = _empty(x, (N, K), other) if need_dw else None
    db = _empty(x, (N,), other) if need_db else None
    _call("poot_linear_backward", dev,
          _PACK_LINEAR_BWD.pack(dy.data_ptr(), x.data_ptr(), pw, _ptr(dx), _ptr(dw), _ptr(db), M, N, K, ld_dy, ldx,
                                code), handle)
    return dx, dw, db


_GRAD_CODES = {torch.float16: GRAD_F16, torch.bfloat16: GRAD_BF16, torch.float32: GRAD_F32}


def _refuse_grad(g, d, i, device):
    """Raises what clip_grad_norm found wrong with pair i."""
    for name, t in (("grads", g), ("out", d)):
        if not isinstance(t, torch.Tensor) or t.dtype not in _GRAD_CODES:
            raise TypeError(f"{name}[{i}] must be a float16, bfloat16 or float32 tensor")
        if t.get_device() != device or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be a contiguous CUDA tensor on the device of the first")
    if d.dtype != g.dtype or d.shape != g.shape:
        raise ValueError(f"out[{i}] must have the shape and dtype of grads[{i}]")


def clip_grad_norm(grads, max_norm: float, *, out=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm.

    grads: a sequence of contiguous CUDA tensors of one device (float16,
    bfloat16 or float32, any mixture), clipped in place; with ``out``, a
    sequence of tensors of the same shapes and dtypes, the results go there
    instead.  The norm, over all tensors together, is a float32 scalar tensor
    on the device (the call does not synchronise).
    """
    grads = list(grads)
    dsts = grads if out is None else list(out)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    if len(dsts) != len(grads):
        raise ValueError(f"out must hold {len(grads)} tensors, got {len(dsts)}")
    # one pass per property over the whole list, in the interpreter's own loops
    T = torch.Tensor
    n = len(grads)
    try:
        dtypes, shapes = [g.dtype for g in grads], [g.shape for g in grads]
        devices = list(map(T.get_device, grads))
        codes = [_GRAD_CODES[t] for t in dtypes]
        src, sizes = list(map(T.data_ptr, grads)), map(T.numel, grads)
        ok = devices[0] >= 0 and devices.count(devices[0]) == n and all(map(T.is_contiguous, grads))
        dst = src
        if ok and out is not None:
            dst = list(map(T.data_ptr, dsts))
            ok = (shapes == [d.shape for d in dsts] and dtypes == [d.dtype for d in dsts]
                  and devices == list(map(T.get_device, dsts)) and all(map(T.is_contiguous, dsts)))
    except (TypeError, AttributeError, KeyError, RuntimeError):
        ok = False
    if not ok:
        device = grads[0].get_device() if isinstance(grads[0], T) else -1
        for i, (g, d) in enumerate(zip(grads, dsts)):
            _refuse_grad(g, d, i, device)
    device = devices[0]
    table = b"".join(map(_PACK_GRAD.pack, src, dst, sizes, codes))
    handle, other = _stream(device, stream)
    first = grads[0]
    norm = _empty(first, (), other, torch.float32)
    _call("poot_clip_grad_norm", device, table, n, max_norm, norm.data_ptr(), handle)
    return norm

"""The feed-forward C ABI on the CPU: exports, argument checks, refusals.

Argument errors are found before any CUDA call, so no GPU is needed; the
addresses are never dereferenced.
"""
import os
import re

import pytest
import torch

import linear_fp16_gb300 as L
from linear_fp16_gb300 import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "poot_ffn.h")).read()
A = [0x1000_0000_0 * (i + 1) for i in range(12)]   # far apart, 256-byte aligned
INV, MIS = L.POOT_ERR_INVALID_ARG, L.POOT_ERR_MISALIGNED


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"POOT_API\s+int\s+(poot_\w+)\s*\(", HEADER))
    assert names == set(ffn.EXPORTS)
    lib = ffn.load_library()
    assert all(hasattr(lib, n) and hasattr(L, n) for n in names)


def test_constants_match_the_header():
    src = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    vals = dict(re.findall(r"\bPOOT_([A-Z0-9_]+)\s*=\s*(\d+)", src))
    assert len(vals) == 6
    for name, v in vals.items():
        assert getattr(ffn, name) == int(v), name


def gated(**kw):
    d = dict(x=A[0], wg=A[1], wu=A[2], bg=A[3], bu=A[4], h=A[5], g=A[6], u=A[7], M=4, N=16, K=8, ldx=0, dtype=0,
             activation=0)
    d.update(kw)
    return L.poot_gated_linear(L.GatedLinearArgs(**d), 0)


def gated_bwd(**kw):
    d = dict(dh=A[0], x=A[1], wg=A[2], wu=A[3], g=A[4], u=A[5], dx=A[6], dwg=A[7], dwu=A[8], dbg=A[9], dbu=A[10],
             M=4, N=16, K=8, dtype=0, activation=0)
    d.update(kw)
    return L.poot_gated_linear_backward(L.GatedLinearBackwardArgs(**d), 0)


def linear_bwd(**kw):
    d = dict(dy=A[0], x=A[1], w=A[2], dx=A[3], dw=A[4], db=A[5], M=4, N=16, K=8, dtype=0)
    d.update(kw)
    return L.poot_linear_backward(L.LinearBackwardArgs(**d), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-1), INV), (dict(M=1 << 31), INV), (dict(K=1 << 31), INV),
    (dict(ldx=7), INV), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(activation=3), INV),
    (dict(activation=-1), INV), (dict(x=0), INV), (dict(wg=0), INV), (dict(wu=0), INV), (dict(h=0), INV),
    (dict(g=0), INV), (dict(u=0), INV),                       # only one of the two
    (dict(x=A[0] + 1), MIS), (dict(wu=A[2] + 1), MIS), (dict(bg=A[3] + 1), MIS), (dict(h=A[5] + 1), MIS),
    (dict(g=A[6] + 1), MIS),
    (dict(h=A[0] + 8), INV), (dict(h=A[1] - 2), INV), (dict(g=A[5] + 2), INV), (dict(u=A[4]), INV),
    (dict(ldx=1000, h=A[0] + 2 * 3 * 1000), INV),             # inside x's last row
])
def test_gated_refusals(kw, code):
    assert gated(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(N=1 << 31), INV), (dict(ldx=7), INV), (dict(ld_dh=15), INV), (dict(ld_g=15), INV),
    (dict(ld_u=15), INV), (dict(dtype=2), INV), (dict(activation=5), INV), (dict(dh=0), INV), (dict(x=0), INV),
    (dict(wg=0), INV), (dict(wu=0), INV), (dict(g=0), INV), (dict(u=0), INV), (dict(dh=A[0] + 1), MIS),
    (dict(dwg=A[7] + 1), MIS), (dict(dx=A[1]), INV), (dict(dwu=A[7]), INV), (dict(dbg=A[10] + 2), INV),
    (dict(dwg=A[4] + 4), INV),
])
def test_gated_backward_refusals(kw, code):
    assert gated_bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(K=-1), INV), (dict(ldx=7), INV), (dict(ld_dy=15), INV), (dict(dtype=3), INV), (dict(dy=0), INV),
    (dict(x=0), INV), (dict(w=0), INV), (dict(w=A[2] + 1), MIS), (dict(db=A[5] + 1), MIS), (dict(dx=A[0]), INV),
    (dict(dw=A[2] + 2), INV), (dict(db=A[4] + 4), INV),
])
def test_linear_backward_refusals(kw, code):
    assert linear_bwd(**kw) == code


def test_null_arguments():
    assert L.poot_gated_linear(None, 0) == INV
    assert L.poot_gated_linear_backward(None, 0) == INV
    assert L.poot_linear_backward(None, 0) == INV


def test_nothing_to_do_needs_no_device():
    assert gated(M=0, x=0, h=0, g=0, u=0) == L.POOT_OK
    assert gated(N=0, wg=0, wu=0, h=0, g=0, u=0) == L.POOT_OK
    none = dict(dx=0, dwg=0, dwu=0, dbg=0, dbu=0)
    assert gated_bwd(**none) == L.POOT_OK
    assert linear_bwd(dx=0, dw=0, db=0) == L.POOT_OK


def test_inputs_of_unwanted_outputs_may_be_null():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # every check passes; the device query then fails without a GPU
    assert gated_bwd(x=0, dwg=0, dwu=0) == L.POOT_ERR_CUDA
    assert gated_bwd(wg=0, wu=0, dx=0) == L.POOT_ERR_CUDA
    assert linear_bwd(x=0, dw=0) == L.POOT_ERR_CUDA
    assert linear_bwd(w=0, dx=0) == L.POOT_ERR_CUDA
    assert gated(bg=0, bu=0, g=0, u=0) == L.POOT_ERR_CUDA


def clip(tensors, max_norm=1.0, norm=A[11], count=None):
    arr = (L.GradTensor * max(1, len(tensors)))(*[L.GradTensor(*t) for t in tensors])
    return L.poot_clip_grad_norm(arr, len(tensors) if count is None else count, max_norm, norm, 0)


@pytest.mark.parametrize("tensors,kw,code", [
    ([(A[0], A[1], 8, 3)], {}, INV), ([(A[0], A[1], -1, 0)], {}, INV), ([(A[0], A[1], (1 << 40) + 1, 0)], {}, INV),
    ([(0, A[1], 8, 0)], {}, INV), ([(A[0], 0, 8, 0)], {}, INV), ([(A[0], A[0], 8, 0)], dict(max_norm=-1.0), INV),
    ([(A[0], A[0], 8, 0)], dict(max_norm=float("nan")), INV), ([(A[0], A[0], 8, 0)], dict(norm=0), INV),
    ([(A[0], A[0], 8, 0)], dict(norm=A[11] + 2), MIS), ([(A[0], A[0], 8, 0)], dict(count=-1), INV),
    ([(A[0] + 1, A[1], 8, 0)], {}, MIS), ([(A[0] + 2, A[1], 8, 2)], {}, MIS), ([(A[0], A[1] + 2, 8, 2)], {}, MIS),
    ([(A[0], A[0] + 4, 8, 0)], {}, INV),                               # dst runs into its own src
    ([(A[0], A[1], 8, 0), (A[2], A[1] + 8, 8, 0)], {}, INV),           # two dst overlap
    ([(A[0], A[0], 8, 0), (A[0] + 8, A[2], 8, 0)], {}, INV),           # a src over another's dst
    ([(A[0], A[1], 1000, 0), (A[2], A[0] + 16, 8, 0)], {}, INV),       # dst inside another's src
    ([(A[0], A[0], 8, 0)], dict(norm=A[0] + 4), INV),                  # the norm inside a tensor
])
def test_clip_refusals(tensors, kw, code):
    assert clip(tensors, **kw) == code


def test_clip_accepts_shared_sources():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert clip([(A[0], A[1], 8, 0), (A[0], A[2], 8, 0), (0, 0, 0, 2)]) == L.POOT_ERR_CUDA


def test_tensor_calls_refuse_what_they_cannot_take():
    t = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        L.gated_linear(t, t, t)                      # CPU tensors
    with pytest.raises(TypeError):
        L.gated_linear(t.float(), t, t)
    with pytest.raises(ValueError):
        L.linear_backward(t, t, t)
    with pytest.raises(TypeError):
        L.clip_grad_norm([t.double()], 1.0)
    with pytest.raises(ValueError):
        L.clip_grad_norm([t], 1.0)
    with pytest.raises(ValueError):
        L.clip_grad_norm([], 1.0)

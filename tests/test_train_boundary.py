"""The training operators' C ABI on the CPU: exports, argument checks, refusals.

Argument errors are found before any CUDA call, so no GPU is needed; the
addresses are never dereferenced.
"""
import os
import re

import pytest
import torch

import linear_fp16_gb300 as L
from linear_fp16_gb300 import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "poot_train.h")).read()
A = [0x1000_0000_0 * (i + 1) for i in range(12)]   # far apart, 256-byte aligned
INV, MIS = L.POOT_ERR_INVALID_ARG, L.POOT_ERR_MISALIGNED


def test_every_declared_symbol_is_exported_and_bound():
    names = set(re.findall(r"POOT_API\s+int\s+(poot_\w+)\s*\(", HEADER))
    assert names == set(train.EXPORTS)
    lib = train.load_library()
    assert all(hasattr(lib, n) and hasattr(L, n) for n in names)


def test_structures_match_the_header():
    src = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    for body, name in re.findall(r"typedef struct \w+ \{(.*?)\} (\w+);", src, flags=re.S):
        fields = [f.strip(" *") for line in body.split(";") if line.strip()
                  for f in re.sub(r"^\s*(const\s+)?\w+", "", line.strip()).split(",")]
        cls = getattr(L, "".join(part.capitalize() for part in name[len("poot_"):].split("_")))
        assert [f for f, _ in cls._fields_] == fields, name


def loss(**kw):
    d = dict(x=A[0], w=A[1], b=A[2], target=A[3], loss=A[4], lse=A[5], M=4, V=16, K=8, ldx=0, ignore_index=-100, dtype=0)
    d.update(kw)
    return L.poot_linear_cross_entropy(L.LinearCrossEntropyArgs(**d), 0)


def loss_bwd(**kw):
    d = dict(dloss=A[0], x=A[1], w=A[2], b=A[3], target=A[4], lse=A[5], dx=A[6], dw=A[7], db=A[8], M=4, V=16, K=8,
             ldx=0, dloss_stride=1, ignore_index=-100, dtype=0)
    d.update(kw)
    return L.poot_linear_cross_entropy_backward(L.LinearCrossEntropyBackwardArgs(**d), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(V=-1), INV), (dict(K=-1), INV), (dict(M=1 << 31), INV), (dict(V=1 << 31), INV),
    (dict(V=0), INV), (dict(ldx=7), INV), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(x=0), INV),
    (dict(w=0), INV), (dict(target=0), INV), (dict(loss=0), INV), (dict(x=A[0] + 1), MIS), (dict(w=A[1] + 1), MIS),
    (dict(b=A[2] + 1), MIS), (dict(target=A[3] + 4), MIS), (dict(loss=A[4] + 2), MIS), (dict(lse=A[5] + 2), MIS),
    (dict(loss=A[0] + 8), INV), (dict(lse=A[3] + 16), INV), (dict(lse=A[4] + 12), INV), (dict(loss=A[2]), INV),
    (dict(M=1 << 30, K=1 << 30), INV), (dict(ldx=1 << 50), INV),
])
def test_loss_refusals(kw, code):
    assert loss(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(V=1 << 31), INV), (dict(V=0), INV), (dict(ldx=7), INV), (dict(dtype=5), INV),
    (dict(dloss_stride=-1), INV), (dict(dloss_stride=1 << 50), INV), (dict(dloss=0), INV), (dict(x=0), INV),
    (dict(w=0), INV), (dict(target=0), INV), (dict(lse=0), INV), (dict(dloss=A[0] + 2), MIS), (dict(x=A[1] + 1), MIS),
    (dict(target=A[4] + 4), MIS), (dict(lse=A[5] + 1), MIS), (dict(dx=A[6] + 1), MIS), (dict(db=A[8] + 1), MIS),
    (dict(dx=A[1]), INV), (dict(dw=A[2] + 2), INV), (dict(db=A[7] + 4), INV), (dict(dw=A[4]), INV),
    (dict(db=A[3]), INV), (dict(dloss_stride=1000, dx=A[0] + 4 * 3 * 1000), INV),
])
def test_loss_backward_refusals(kw, code):
    assert loss_bwd(**kw) == code


def test_null_arguments():
    assert L.poot_linear_cross_entropy(None, 0) == INV
    assert L.poot_linear_cross_entropy_backward(None, 0) == INV


def test_nothing_to_do_needs_no_device():
    assert loss(M=0, x=0, target=0, loss=0, lse=0) == L.POOT_OK
    assert loss(M=0, V=0, x=0, w=0, target=0, loss=0, lse=0) == L.POOT_OK
    assert loss_bwd(dx=0, dw=0, db=0) == L.POOT_OK
    assert loss_bwd(K=0, db=0) == L.POOT_OK


def test_optional_pointers_may_be_null():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # every check passes; the device query then fails without a GPU
    assert loss(b=0, lse=0) == L.POOT_ERR_CUDA
    assert loss(K=0, x=0, w=0) == L.POOT_ERR_CUDA
    assert loss_bwd(b=0, dx=0, db=0) == L.POOT_ERR_CUDA
    assert loss_bwd(dw=0, dloss_stride=0) == L.POOT_ERR_CUDA
    assert loss_bwd(M=0, x=0, dloss=0, target=0, lse=0) == L.POOT_ERR_CUDA


def test_tensor_calls_refuse_what_they_cannot_take():
    x, w, t = torch.zeros(4, 8).half(), torch.zeros(16, 8).half(), torch.zeros(4, dtype=torch.int64)
    lse = torch.zeros(4)
    with pytest.raises(ValueError):
        L.linear_cross_entropy(x, w, t)                # CPU tensors
    with pytest.raises(TypeError):
        L.linear_cross_entropy(x.float(), w, t)
    with pytest.raises(TypeError):
        L.linear_cross_entropy([1.0], w, t)
    with pytest.raises(ValueError):
        L.linear_cross_entropy_backward(lse, x, w, t, lse)


B = A[0]
NAN, INF = float("nan"), float("inf")


def tensors(*changes):
    """Parameters of 8 elements far apart, with the changes made to each."""
    out = []
    for i, kw in enumerate(changes):
        base = B + i * 0x1000_0000
        d = dict(param=base, grad=base + 0x100_0000, m=base + 0x200_0000, v=base + 0x300_0000, m_scale=base + 0x400_0000,
                 v_scale=base + 0x500_0000, copy=0, n=8, weight_decay=0.01, param_dtype=2, grad_dtype=1, copy_dtype=1)
        d.update(kw)
        out.append(L.AdamwTensor(**d))
    return (L.AdamwTensor * max(1, len(out)))(*out)


def adamw(*changes, **kw):
    d = dict(tensors=tensors(*changes), count=len(changes), step=1, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
             grad_scale=1.0, bits=32)
    d.update(kw)
    return L.poot_adamw_step(L.AdamwArgs(**d), 0)


@pytest.mark.parametrize("changes,kw,code", [
    ([{}], dict(count=-1), INV), ([{}], dict(tensors=None), INV), ([{}], dict(bits=16), INV),
    ([{}], dict(beta1=1.0), INV), ([{}], dict(beta1=-0.1), INV), ([{}], dict(beta2=1.0), INV), ([{}], dict(beta2=NAN), INV),
    ([{}], dict(eps=-1e-8), INV), ([{}], dict(eps=NAN), INV), ([{}], dict(lr=-1.0), INV), ([{}], dict(lr=INF), INV),
    ([{}], dict(step=0), INV), ([{}], dict(grad_scale=INF), INV), ([{}], dict(lr_device=A[3] + 2), MIS),
    ([{}], dict(step_device=A[3] + 4), MIS), ([{}], dict(grad_scale_device=A[3] + 1), MIS),
    ([dict(n=-1)], {}, INV), ([dict(n=(1 << 40) + 1)], {}, INV), ([dict(param_dtype=3)], {}, INV),
    ([dict(grad_dtype=-1)], {}, INV), ([dict(weight_decay=-1.0)], {}, INV), ([dict(weight_decay=NAN)], {}, INV),
    ([dict(param=0)], {}, INV), ([dict(grad=0)], {}, INV), ([dict(m=0)], {}, INV), ([dict(v=0)], {}, INV),
    ([dict(m_scale=0)], dict(bits=8), INV), ([dict(v_scale=0)], dict(bits=8), INV),
    ([dict(copy=B + 0x600_0000, copy_dtype=2)], {}, INV), ([dict(copy=B + 0x600_0000, param_dtype=1)], {}, INV),
    ([dict(param=B + 2)], {}, MIS), ([dict(grad=B + 0x100_0001)], {}, MIS), ([dict(m=B + 0x200_0002)], {}, MIS),
    ([dict(copy=B + 0x600_0001)], {}, MIS), ([dict(m_scale=B + 0x400_0002)], dict(bits=8), MIS),
    ([dict(grad=B + 16)], {}, INV),                                     # inside the parameter
    ([dict(v=B + 0x200_0000)], {}, INV),                                # m and v the same
    ([dict(m=B + 28)], {}, INV), ([dict(v_scale=B + 0x200_0004)], dict(bits=8), INV),
    ([{}, dict(param=B)], {}, INV),                                     # one parameter twice
    ([{}, dict(param=B + 0x100_0000)], {}, INV),                        # a parameter that is another's gradient
    ([{}, dict(copy=B + 0x100_0000)], {}, INV),                         # a copy over another's gradient
    ([{}], dict(step_device=B + 0x200_0000), INV), ([{}], dict(lr_device=B + 4), INV),
])
def test_adamw_refusals(changes, kw, code):
    assert adamw(*changes, **kw) == code


def test_adamw_takes():
    assert L.poot_adamw_step(None, 0) == INV
    assert adamw() == L.POOT_OK and adamw(dict(n=0, param=0, grad=0, m=0, v=0)) == L.POOT_OK
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    # every check passes; the device query then fails without a GPU
    assert adamw({}, {}) == L.POOT_ERR_CUDA
    assert adamw(dict(grad=B + 0x100_0000), dict(grad=B + 0x100_0000)) == L.POOT_ERR_CUDA   # one gradient for two
    assert adamw(dict(m=B + 0x200_0001, v=B + 0x300_0003), bits=8) == L.POOT_ERR_CUDA       # codes anywhere
    assert adamw({}, step=0, step_device=A[3], lr=NAN, lr_device=A[4], grad_scale=NAN,
                 grad_scale_device=A[5]) == L.POOT_ERR_CUDA


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INV), (dict(m=0), INV), (dict(v_scale=0), INV), (dict(m_out=0), INV), (dict(m_scale=A[2] + 1), MIS),
    (dict(v_out=A[5] + 2), MIS), (dict(m_out=A[0]), INV), (dict(v_out=A[4] + 16), INV), (dict(n=0, m=0), L.POOT_OK),
])
def test_adamw_values_refusals(kw, code):
    d = dict(m=A[0], v=A[1], m_scale=A[2], v_scale=A[3], m_out=A[4], v_out=A[5], n=8)
    d.update(kw)
    assert L.poot_adamw_values((L.AdamwCodes * 1)(L.AdamwCodes(**d)), 1, 0) == code


def test_adamw_calls_refuse_what_they_cannot_take():
    p = [torch.zeros(4, 8)]
    for bits in (32, 8):
        state = L.adamw_state(p, bits=bits)
        assert state.bits == bits and [t.shape for t in state.m] == [(4, 8)]
        with pytest.raises(ValueError):
            L.adamw_step(p, p, state, step=1)          # CPU tensors
    assert state.m[0].dtype == torch.int8 and state.v[0].dtype == torch.uint8 and state.m_scale[0].shape == (1,)
    with pytest.raises(ValueError):
        L.adamw_step([], [], state, step=1)
    with pytest.raises(ValueError):
        L.adamw_step(p, [], state, step=1)
    with pytest.raises(ValueError):
        L.adamw_state(p, bits=16)

"""Gradients with nothing to compute, or only part of it, through the C calls
(torch hands NULL for an empty tensor, a C caller need not)."""
import pytest
import torch

import linear_fp16_gb300 as L
from tests import ffn_ref as R

A = [0x1000_0000_0 * (i + 1) for i in range(12)]   # never dereferenced
F16 = torch.float16
DEV = "cuda:0"


def _gated_bwd(**kw):
    d = dict(dh=A[0], x=A[1], wg=A[2], wu=A[3], g=A[4], u=A[5], dx=A[6], dwg=A[7], dwu=A[8], M=4, N=16, K=0)
    d.update(kw)
    return L.poot_gated_linear_backward(L.GatedLinearBackwardArgs(**d), 0)


@pytest.mark.parametrize("kw", [{}, dict(dx=0), dict(dwg=0, dwu=0), dict(dwu=0), dict(M=0), dict(N=0), dict(dtype=1)])
def test_gated_backward_without_columns_and_bias_gradients(kw):
    assert _gated_bwd(**kw) == L.POOT_OK


@pytest.mark.parametrize("kw", [{}, dict(dx=0), dict(dw=0), dict(M=0)])
def test_linear_backward_without_columns_and_bias_gradient(kw):
    d = dict(dy=A[0], x=A[1], w=A[2], dx=A[3], dw=A[4], db=0, M=4, N=16, K=0)
    d.update(kw)
    assert L.poot_linear_backward(L.LinearBackwardArgs(**d), 0) == L.POOT_OK


def test_argument_errors_come_first():
    assert _gated_bwd(dh=0) == L.POOT_ERR_INVALID_ARG
    assert _gated_bwd(dwu=A[0] + 1) == L.POOT_ERR_MISALIGNED


def _inputs(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(F16)
    return dict(dh=n(M, N), x=n(M, K), wg=n(N, K), wu=n(N, K), g=n(M, N), u=n(M, N))


@pytest.mark.gpu
@pytest.mark.parametrize("outs", [("dbg", "dbu"), ("dbg",), ("dbu",), ("dx", "dwg", "dbu"), ("dx", "dwg", "dwu")])
def test_gated_backward_without_columns_on_a_device(outs):
    M, N = 70, 40
    t = {k: v.to(DEV) for k, v in _inputs(M, N, 0, 5).items()}
    out = {k: torch.full((N,), float("nan"), dtype=F16, device=DEV) for k in outs}
    rc = L.poot_gated_linear_backward(L.GatedLinearBackwardArgs(
        **{k: v.data_ptr() for k, v in t.items()}, **{k: v.data_ptr() for k, v in out.items()}, M=M, N=N, K=0), 0)
    torch.cuda.synchronize()
    assert rc == L.POOT_OK and L.poot_linear_device_status(0) == L.POOT_OK
    (dg, du), (eg, eu) = R.gate_grad64(t["dh"].cpu(), t["g"].cpu(), t["u"].cpu(), "silu")
    for name, d, e in (("dbg", dg, eg), ("dbu", du, eu)):
        if name in out:
            R.check(out[name], d.sum(0), e.sum(0) + (M + 16) * 2.0 ** -24 * d.abs().sum(0), name)
    for name in set(outs) - {"dbg", "dbu"}:
        assert torch.isnan(out[name]).all(), name    # no element of it to write


@pytest.mark.gpu
@pytest.mark.parametrize("outs", [("dwg",), ("dwu",), ("dbg",), ("dbu",), ("dwu", "dbg"), ("dx", "dwg", "dbu")])
def test_any_subset_of_the_gradients(outs):
    """One of dwg and dwu, one of dbg and dbu: the bits of the call for all."""
    M, N, K = 90, 136, 72
    t = {k: v.to(DEV) for k, v in _inputs(M, N, K, 6).items()}
    shapes = dict(dx=(M, K), dwg=(N, K), dwu=(N, K), dbg=(N,), dbu=(N,))

    def run(names):
        out = {k: torch.full(shapes[k], float("nan"), dtype=F16, device=DEV) for k in names}
        rc = L.poot_gated_linear_backward(L.GatedLinearBackwardArgs(
            **{k: v.data_ptr() for k, v in t.items()}, **{k: v.data_ptr() for k, v in out.items()}, M=M, N=N, K=K), 0)
        torch.cuda.synchronize()
        assert rc == L.POOT_OK and L.poot_linear_device_status(0) == L.POOT_OK
        return out
    full = run(tuple(shapes))
    some = run(outs)
    # A plan of fewer products may split its sums otherwise: two FP32 orders of
    # sums whose terms' magnitudes add up to less than 200 (2 (90 / 16 + 64) 2^-23 200
    # = 2^-8.1), then one rounding each, at most one spacing apart
    for k in outs:
        d = (some[k].double() - full[k].double()).abs()
        assert bool((d <= 2.0 ** -10 * full[k].double().abs() + 2.0 ** -8).all()), k

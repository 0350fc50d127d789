"""Sizes and pitches at the ends of their ranges, on the C calls.

Addresses are not dereferenced in the CPU tests: a call that passes its checks
ends at the device query there.
"""
import os
import re

import pytest
import torch

import linear_fp16_gb300 as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x100_0000_0000_00 * (i + 1) for i in range(12)]   # 2^44 bytes apart
TOP = int(re.search(r"#define POOT_FFN_MAX_SIZE (\d+)", open(os.path.join(ROOT, "include", "poot_ffn.h")).read())[1])
INV = L.POOT_ERR_INVALID_ARG
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


def gated(**kw):
    d = dict(x=A[0], wg=A[1], wu=A[2], h=A[5], M=4, N=16, K=8)
    d.update(kw)
    return L.poot_gated_linear(L.GatedLinearArgs(**d), 0)


def gated_bwd(**kw):
    d = dict(dh=A[0], x=A[1], wg=A[2], wu=A[3], g=A[4], u=A[5], dx=A[6], dwg=A[7], dwu=A[8], M=4, N=16, K=8)
    d.update(kw)
    return L.poot_gated_linear_backward(L.GatedLinearBackwardArgs(**d), 0)


def linear_bwd(**kw):
    d = dict(dy=A[0], x=A[1], w=A[2], dx=A[3], dw=A[4], db=A[5], M=4, N=16, K=8)
    d.update(kw)
    return L.poot_linear_backward(L.LinearBackwardArgs(**d), 0)


CALLS = [gated, gated_bwd, linear_bwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dim", ["M", "N", "K"])
def test_sizes_that_32_bit_index_arithmetic_cannot_round_up(call, dim):
    """A size above 2^31 - 1024 plus a tile, a span or a warp's share of K passed
    2^31: in the GEMVs a warp's range of K then began below zero."""
    for size in (TOP + 1, (1 << 31) - 1024, (1 << 31) - 8, (1 << 31) - 1):
        assert call(**{dim: size}) == INV, size


@no_gpu
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dim", ["M", "N", "K"])
def test_the_largest_size_passes_the_checks(call, dim):
    assert call(**{dim: TOP, **{d: 1 for d in "MNK" if d != dim}}) == L.POOT_ERR_CUDA


@pytest.mark.gpu
@pytest.mark.parametrize("K", [TOP, TOP - 3])
def test_rows_of_nearly_31_bits(K):
    """A decode row over the largest K (16-byte rows, and any alignment): all
    but a few elements zero, small integers there, so that g and u are exact."""
    F16, dev = torch.float16, "cuda:0"
    at = [0, 7, 64, K // 16 * 7 + 5, K // 2, K // 16 * 15, K - 513, K - 2, K - 1]
    x = torch.zeros(1, K, dtype=F16, device=dev)
    w = [torch.zeros(2, K, dtype=F16, device=dev) for _ in range(2)]
    for i, k in enumerate(at):
        x[0, k] = i + 1
        for j in range(2):
            w[j][0, k] = j + 1
            w[j][1, k] = (i % 3) - 1 + j
    _, g, u = L.gated_linear(x, *w, save=True)
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    n = len(at)
    for j, got in enumerate((g, u)):
        assert got.tolist() == [[float((j + 1) * n * (n + 1) // 2), float(sum((i + 1) * (i % 3 - 1 + j) for i in range(n)))]]


PITCHES = [(gated, "ldx"), (gated_bwd, "ldx"), (gated_bwd, "ld_dh"), (gated_bwd, "ld_g"), (gated_bwd, "ld_u"),
           (linear_bwd, "ldx"), (linear_bwd, "ld_dy")]


@pytest.mark.parametrize("call,ld", PITCHES)
def test_pitches_that_no_matrix_has(call, ld):
    """Byte counts of such rows wrapped, and with them the overlap checks."""
    for v in (1 << 50, 1 << 61, 1 << 62, (1 << 63) - 1):
        assert call(**{ld: v}) == INV, v
    assert call(**{ld: -1}) == INV


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("big", ["MN", "MK", "NK"])
def test_matrices_beyond_any_address_space(call, big):
    assert call(**{d: TOP if d in big else 1 for d in "MNK"}) == INV


@no_gpu
@pytest.mark.parametrize("call,ld", PITCHES)
def test_a_single_row_has_no_pitch(call, ld):
    assert call(**{"M": 1, ld: (1 << 63) - 1}) == L.POOT_ERR_CUDA


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(48, 40), (45, 37)])
def test_gradients_of_a_single_row_at_any_pitch(N, K):
    dev = "cuda:0"
    g = torch.Generator().manual_seed(N)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).half()
    dy, x, w = ints(1, N), ints(1, K), ints(N, K)
    t = [v.to(dev) for v in (dy, x, w)]
    out = [torch.empty(s, dtype=torch.float16, device=dev) for s in ((1, K), (N, K), (N,))]
    for ld in (0, 1 << 20, (1 << 20) + 1, 1 << 45):
        for o in out:
            o.fill_(float("nan"))
        rc = L.poot_linear_backward(L.LinearBackwardArgs(
            dy=t[0].data_ptr(), x=t[1].data_ptr(), w=t[2].data_ptr(), dx=out[0].data_ptr(), dw=out[1].data_ptr(),
            db=out[2].data_ptr(), M=1, N=N, K=K, ld_dy=ld, ldx=ld), 0)
        torch.cuda.synchronize()
        assert rc == L.POOT_OK and L.poot_linear_device_status(0) == L.POOT_OK, ld
        for o, r in zip(out, (dy.double() @ w.double(), dy.double().T @ x.double(), dy.double()[0])):
            assert torch.equal(o.cpu(), r.half()), ld

"""Sums over more elements than one chunk of the tensor core's accumulator (8192
in binary16, 32768 in bfloat16): exact on small integers, and free of the truncation's drift on sums of
one sign.  The plans named are those of 152 SMs.
"""
import pytest
import torch

import linear_fp16_gb300 as L
from tests import ffn_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(g, shape, dt, hi=1):
    return torch.randint(-hi, hi + 1, shape, generator=g, device=DEV, dtype=torch.int8).to(dt)


def _ok():
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK


def _mm(a, b):
    """a b for integers of FP32 sums below 2^24, in 64 bits by slices of the long side."""
    out = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=DEV)
    for k in range(0, a.shape[1], 8192):
        out += a[:, k:k + 8192].double() @ b[k:k + 8192].double()
    return out


# single CTAs: narrow tiles, split in 16 ranges of several chunks (whole rows, odd rows); wide
# ones the same; CTA pairs, unsplit, five chunks
@pytest.mark.parametrize("M,N,K,dt", [(64, 256, 524288, F16), (33, 72, 400001, F16), (300, 264, 400000, F16),
                                      (1024, 4096, 40000, F16), (2048, 1000, 40000, F16), (1024, 4096, 100000, BF16),
                                      (64, 256, 2200000, BF16)])
def test_gated_linear_over_long_rows(M, N, K, dt):
    g = _gen(K)
    x, wg, wu = _ints(g, (M, K), dt), _ints(g, (N, K), dt), _ints(g, (N, K), dt)
    bg, bu = _ints(g, (N,), dt, 50), _ints(g, (N,), dt, 50)
    h, gs, us = L.gated_linear(x, wg, wu, bg, bu, save=True)
    _ok()
    rows = torch.arange(0, M, max(1, M // 200), device=DEV)
    gd, ud = _mm(x[rows], wg.T) + bg.double(), _mm(x[rows], wu.T) + bu.double()
    assert torch.equal(gs[rows], gd.to(dt)) and torch.equal(us[rows], ud.to(dt))
    # h from exact sums, with the activation's bound of ffn_ref; products beyond
    # binary16's range are infinities (at 65520 and above, to the bound)
    a = R.act64("silu", gd)
    ref, err = (a * ud).cpu(), (R.ACT_ERR * gd.abs() * ud.abs() + 2.0 ** -22 * (a * ud).abs()).cpu()
    got, top = h[rows].cpu(), 65520.0 if dt == F16 else float("inf")
    inside = ref.abs() + err < top
    R.check(got[inside], ref[inside], err[inside], "h")
    beyond = ref.abs() - err > top
    assert torch.equal(got[beyond].double(), torch.sign(ref[beyond]) * float("inf"))


# dx over N, dW over M: pairs and single CTAs, split and unsplit, one and both of several chunks
@pytest.mark.parametrize("M,N,K,dt", [(2048, 40000, 2048, F16), (40000, 4096, 1032, F16), (130, 400000, 70, F16),
                                      (40000, 264, 520, F16), (20000, 20000, 264, F16), (2048, 300000, 1024, BF16),
                                      (1100000, 264, 520, BF16), (300000, 4096, 264, BF16)])
def test_linear_backward_over_long_sums(M, N, K, dt):
    g = _gen(M + K)
    dy, x, w = _ints(g, (M, N), dt), _ints(g, (M, K), dt), _ints(g, (N, K), dt)
    dx, dw, db = L.linear_backward(dy, x, w)
    _ok()
    rows = torch.arange(0, M, max(1, M // 100), device=DEV)
    cols = torch.arange(0, N, max(1, N // 100), device=DEV)
    assert torch.equal(dx[rows], _mm(dy[rows], w).to(dt))
    assert torch.equal(dw[cols], _mm(dy.T[cols].contiguous(), x).to(dt))
    assert torch.equal(db, dy.double().sum(0).to(dt))


@pytest.mark.parametrize("M,N,K,dt", [(40000, 1024, 1024, F16), (400000, 200, 136, F16), (2048, 20000, 2048, F16),
                                      (256, 40000, 1000, F16), (300000, 1024, 1024, BF16), (256, 300000, 1000, BF16)])
def test_gated_linear_backward_over_long_sums(M, N, K, dt):
    """g = 64: silu(g) = 64 and silu'(g) = 1 in FP32, so dg and du are integers."""
    gen = _gen(M + N)
    dh, x, wg, wu = _ints(gen, (M, N), dt), _ints(gen, (M, K), dt), _ints(gen, (N, K), dt), _ints(gen, (N, K), dt)
    g, u = torch.full((M, N), 64.0, dtype=dt, device=DEV), _ints(gen, (M, N), dt)
    dx, dwg, dwu, dbg, dbu = L.gated_linear_backward(dh, x, wg, wu, g, u, need_db=True)
    _ok()
    rows = torch.arange(0, M, max(1, M // 100), device=DEV)
    cols = torch.arange(0, N, max(1, N // 100), device=DEV)
    dg, du = dh * u, dh * 64
    assert torch.equal(dx[rows], (_mm(dg[rows], wg) + _mm(du[rows], wu)).to(dt))
    for got, d in ((dwg, dg), (dwu, du)):
        assert torch.equal(got[cols], _mm(d.T[cols].contiguous(), x).to(dt))
    assert torch.equal(dbg, dg.double().sum(0).to(dt)) and torch.equal(dbu, du.double().sum(0).to(dt))


@pytest.mark.parametrize("dt", [F16, BF16])
def test_sums_of_one_sign_do_not_drift(dt):
    """dW over 262144 rows, unsplit, of positive terms; columns of both operands are scaled
    so that the outputs spread over two binades.  Each MMA truncates where it adds
    its 16 products, so a sum in one accumulator comes out low.  The mean
    relative error of 4096 outputs beyond the reference's own rounding stays
    within an eighth of one rounding (2^-14 in binary16, 2^-11 in bfloat16) and
    an eighth of that for the noise of outputs near a rounding boundary."""
    M, N, K = 262144, 4096, 2048
    g = _gen(3)
    rnd = lambda rows, cols: (torch.rand(rows, cols, generator=g, device=DEV, dtype=torch.float32)
                              .mul_(torch.logspace(-3, -2, cols, base=2, device=DEV)).to(dt))
    dy, x = rnd(M, N), rnd(M, K)
    dw = L.linear_backward(dy, x, torch.zeros(N, K, dtype=dt, device=DEV), need_dx=False, need_db=False)[1]
    _ok()
    got, ref = dw[::64, ::32].double(), _mm(dy.T[::64].contiguous(), x[:, ::32])
    p = R.P[dt]
    assert float(((got - ref).abs() / ref).max()) <= 2.0 ** -p + 2.0 ** -(p + 2)
    drift = float(((got - ref.to(dt).double()) / ref).mean())
    assert abs(drift) <= 2.0 ** -(p + 3) + 2.0 ** -(p + 6), drift

"""The activations and their derivatives in their lower tails, relative to
themselves: one rounding of the result and little else.

g = x_m w_n is exact in FP32 and u = 1, so h is act(g) rounded once.  With unit
dh and x the identity, dwu and dwg are du = act(g) and dg = act'(g) as rounded
to the dtype.  Bound: u_p of the result (the rounding) plus 2^-14 of it for the
activation in FP32.  That covers an exponent of at most 134 (in base 2) that
carries up to five roundings of 2^-24 (2^-14.6 times ln 2) and a few ulps more;
a derivative is a sum of two terms, each known to 2^-14 of itself.  Results in the
dtype's subnormal range are also off by half its smallest step.
"""
import math

import pytest
import torch

import linear_fp16_gb300 as L
from tests import ffn_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
ACTS = ("silu", "gelu_tanh", "gelu_erf")


def _act64(act, t):
    """act(t) and the two terms of act'(t), without cancellation."""
    if act == "gelu_erf":
        cdf = 0.5 * torch.special.erfc(-t / math.sqrt(2))
        return t * cdf, cdf, t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    z, dz = t, torch.ones_like(t)
    if act == "gelu_tanh":
        z = math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3)
        dz = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * t * t)
    s = torch.special.expit(z)
    return t * s, s, t * s * torch.special.expit(-z) * dz


def _check(got, ref, err, dt, g, name):
    got = got.cpu().double()
    lim = (2.0 ** -R.P[dt]) * (ref.abs() + err) + err + R.TINY[dt]
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, for g from "
                           f"{float(g[bad].min()):.4g} to {float(g[bad].max()):.4g}, worst "
                           f"{float(((got - ref).abs() / lim)[bad].max()):.3g} times it")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(16, 2048, 16), (5, 1000, 13), (256, 2048, 16), (64, 256, 4096)])
def test_forward_tails(M, N, K, act, dt):
    x = torch.zeros(M, K)
    x[:, 0] = torch.linspace(1, 2, M)
    x[:, 1] = 1.0
    wg, wu = torch.zeros(N, K), torch.zeros(N, K)
    wg[:, 0] = torch.linspace(-52, 4, N)
    wu[:, 1] = 1.0
    x, wg, wu = x.to(dt), wg.to(dt), wu.to(dt)
    h = L.gated_linear(x.to(DEV), wg.to(DEV), wu.to(DEV), activation=act)
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    g = torch.outer(x[:, 0].double(), wg[:, 0].double())
    ref = _act64(act, g)[0]
    _check(h, ref, 2.0 ** -14 * ref.abs(), dt, g, "h")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [2048, 1001])
def test_gradient_tails(N, act, dt):
    M = 64
    one = torch.ones(M, N, dtype=dt)
    g = torch.linspace(-104, 8, M * N).view(N, M).T.contiguous().to(dt)
    eye, w = torch.eye(M, dtype=dt), torch.zeros(N, M, dtype=dt)
    _, dwg, dwu, _, _ = L.gated_linear_backward(one.to(DEV), eye.to(DEV), w.to(DEV), w.to(DEV), g.to(DEV), one.to(DEV),
                                                activation=act, need_dx=False)
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    gd = g.double()
    v, d0, d1 = _act64(act, gd)
    _check(dwu.T, v, 2.0 ** -14 * v.abs(), dt, gd, "du")
    _check(dwg.T, d0 + d1, 2.0 ** -14 * (d0.abs() + d1.abs()), dt, gd, "dg")


@pytest.mark.parametrize("act", ACTS)
def test_the_largest_magnitudes(act):
    """Cubes and squares of g overflow FP32 here: value and slope are the limits'."""
    M, N = 16, 64
    big = torch.tensor([1e3, 1e10, 1e20, 3e38]).repeat(M // 4)
    x = torch.zeros(M, 8)
    x[:, 0], x[:, 1] = big, 1.0
    wg, wu = torch.zeros(N, 8), torch.zeros(N, 8)
    wg[: N // 2, 0], wg[N // 2:, 0], wu[:, 1] = 1.0, -1.0, 1.0
    for rows in (x, x.repeat(8, 1)):
        xb = rows.to(BF16)
        h = L.gated_linear(xb.to(DEV), wg.to(BF16).to(DEV), wu.to(BF16).to(DEV), activation=act).cpu()
        assert torch.equal(h[:, : N // 2], xb[:, :1].expand(-1, N // 2)) and not h[:, N // 2:].any()

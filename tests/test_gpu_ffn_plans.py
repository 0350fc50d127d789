"""The tile plans of training sizes, exact on small integers: CTA pairs on 256
columns with dx and dW dealt over several waves, unsplit; gated CTA pairs with
a split; odd sizes of both.  The plans named are those of 152 SMs.
"""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


def _ints(g, shape, dt, hi=2):
    return torch.randint(-hi, hi + 1, shape, generator=g, device=DEV, dtype=torch.int8).to(dt)


def _gen(*key):
    return torch.Generator(device=DEV).manual_seed(sum((i + 1) * k for i, k in enumerate(key)))


def _ok():
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK


# 128 + 128 tiles over 76 pairs, 128 + 32, 64 + 64; odd sizes, 50 + 68
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 2048), (8000, 2000, 1000), (4096, 4096, 1024), (2500, 4100, 1001)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_linear_backward(M, N, K, dt):
    g = _gen(M, N, K)
    dy, x, w = _ints(g, (M, N), dt), _ints(g, (M, K), dt), _ints(g, (N, K), dt)
    dx, dw, db = L.linear_backward(dy, x, w)
    _ok()
    d = dy.double()
    assert torch.equal(dx, (d @ w.double()).to(dt))
    assert torch.equal(dw, (d.T @ x.double()).to(dt))
    assert torch.equal(db, d.sum(0).to(dt))


# 64 + 128 tiles over 76 pairs, 45 + 160, 48 + 96; odd sizes
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1024), (2304, 4000, 1032), (3000, 3000, 1000), (2304, 4099, 1001)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_gated_linear_backward(M, N, K, dt):
    """g = 64: silu(g) = 64 and silu'(g) = 1 in FP32, so dg and du are integers."""
    gen = _gen(M, N, K, 1)
    dh, x, wg, wu = _ints(gen, (M, N), dt, 1), _ints(gen, (M, K), dt), _ints(gen, (N, K), dt), _ints(gen, (N, K), dt)
    g, u = torch.full((M, N), 64.0, dtype=dt, device=DEV), _ints(gen, (M, N), dt)
    dx, dwg, dwu, dbg, dbu = L.gated_linear_backward(dh, x, wg, wu, g, u, need_db=True)
    _ok()
    dg, du = (dh * u).double(), (dh * 64).double()
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(dt))
    assert torch.equal(dwg, (dg.T @ x.double()).to(dt)) and torch.equal(dwu, (du.T @ x.double()).to(dt))
    assert torch.equal(dbg, dg.sum(0).to(dt)) and torch.equal(dbu, du.sum(0).to(dt))


# pairs: 128 columns split in 4, 8 and 2; 256 columns split in 4, whole and odd
@pytest.mark.parametrize("M,N,K", [(256, 1024, 8192), (512, 256, 8192), (512, 1024, 4096), (768, 512, 4096),
                                   (600, 520, 4100), (601, 521, 4099)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_gated_linear_split_pairs(M, N, K, dt):
    gen = _gen(M, N, K, 2)
    x, wg, wu = _ints(gen, (M, K), dt, 1), _ints(gen, (N, K), dt, 1), _ints(gen, (N, K), dt, 1)
    bg, bu = _ints(gen, (N,), dt, 9), _ints(gen, (N,), dt, 9)
    h, g, u = L.gated_linear(x, wg, wu, bg, bu, save=True)
    _ok()
    gd, ud = x.double() @ wg.double().T + bg.double(), x.double() @ wu.double().T + bu.double()
    assert torch.equal(g, gd.to(dt)) and torch.equal(u, ud.to(dt))
    ref = gd * torch.sigmoid(gd) * ud
    p = 11 if dt == F16 else 8
    # one rounding, 2^-18 |g| of the activation (as in ffn_ref), the smallest step
    lim = 2.0 ** -p * ref.abs() + 1.01 * 2.0 ** -18 * gd.abs() * ud.abs() + 2.0 ** -25
    assert bool(((h.double() - ref).abs() <= lim).all())

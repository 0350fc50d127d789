"""Clipping by the global norm on a GPU against a plain 64-bit form.

The squares are summed in FP32 over at most 64 elements (relative error at
most 64 2^-24) and in FP64 beyond, then one rounding: the norm is within
2^-18 relative of the 64-bit value; a result within that plus one rounding of
its dtype (and the scale's own, 2^-23).
"""
import math

import pytest
import torch

import linear_fp16_gb300 as L
from tests import ffn_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
R.P.setdefault(F32, 24)
R.TINY.setdefault(F32, 2.0 ** -150)


def _check(srcs, outs, norm, max_norm):
    total = math.fsum(float(s.double().square().sum()) for s in srcs)
    ref = math.sqrt(total)
    assert norm.dtype == F32 and norm.dim() == 0
    assert abs(float(norm) - ref) <= 2.0 ** -18 * ref + 2.0 ** -149, (float(norm), ref)
    scale = min(1.0, max_norm / (ref + 1e-6))
    for i, (s, o) in enumerate(zip(srcs, outs)):
        want = s.double() * scale
        R.check(o, want, (2.0 ** -18 + 2.0 ** -23) * want.abs(), f"tensor {i}")


LISTS = {
    "one": [(5, F32)],
    "one_element": [(1, F16)],
    "mixed": [(1000, F16), (17, F32), (0, BF16), (16385, BF16), (8192, F32), (8193, F32), (3, F16)],
    "pieces": [(16384 * 3 + 7, F16), (8192 * 2, F32), (16383, BF16)],
    "many": [(1 + (i * 37) % 300, (F16, BF16, F32)[i % 3]) for i in range(513)],
    "more": [(5, F16)] * 1025,
}


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("max_norm", [0.0, 0.25, 1e5])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip(name, max_norm, in_place):
    g = torch.Generator().manual_seed(len(name))
    srcs = [torch.randn(n, generator=g).to(dt) for n, dt in LISTS[name]]
    dev = [s.to(DEV) for s in srcs]
    out = None if in_place else [torch.full_like(d, float("nan")) for d in dev]
    norm = L.clip_grad_norm(dev, max_norm, out=out)
    torch.cuda.synchronize()
    _check(srcs, dev if in_place else out, norm, max_norm)
    if not in_place:
        assert all(torch.equal(d.cpu(), s) for d, s in zip(dev, srcs))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("so,do", [(0, 0), (1, 1), (3, 3), (1, 2), (0, 7), (5, 0)])
def test_any_element_alignment(dt, so, do):
    n = 40001
    base = torch.randn(n + 16, generator=torch.Generator().manual_seed(so * 8 + do)).to(dt)
    src, dst = base.to(DEV), torch.full((n + 16,), 7.0, dtype=dt, device=DEV)
    norm = L.clip_grad_norm([src[so:so + n]], 1.0, out=[dst[do:do + n]])
    torch.cuda.synchronize()
    _check([base[so:so + n]], [dst[do:do + n]], norm, 1.0)
    assert bool((dst[:do] == 7).all()) and bool((dst[do + n:] == 7).all())


@pytest.mark.parametrize("dt,mag", [(F32, 1e30), (F32, 3e-30), (BF16, 1e30), (BF16, 1e-35), (F16, 6e4), (F16, 6e-8),
                                    (F32, 1e-42)])
def test_squares_outside_the_range_of_fp32(dt, mag):
    n = 5000
    src = (torch.rand(n, generator=torch.Generator().manual_seed(1)) * 0.5 + 0.5).mul(mag).to(dt)
    src[100:4200] = 0
    dev = src.to(DEV)
    out = [torch.empty_like(dev)]
    norm = L.clip_grad_norm([dev], 1.0, out=out)
    torch.cuda.synchronize()
    _check([src], out, norm, 1.0)


def test_all_zero_and_empty():
    z = torch.zeros(70000, dtype=BF16, device=DEV)
    e = torch.zeros(0, dtype=F32, device=DEV)
    assert float(L.clip_grad_norm([z, e], 1.0)) == 0.0 and not z.any()
    assert float(L.clip_grad_norm([e], 1.0)) == 0.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_reach_the_norm(bad):
    src = torch.ones(20000, dtype=BF16)
    src[12345] = bad
    dev = src.to(DEV)
    norm = float(L.clip_grad_norm([dev], 1.0))
    out = dev.cpu()
    if math.isnan(bad):
        assert math.isnan(norm) and torch.isnan(out).all()
    else:
        assert math.isinf(norm) and torch.isnan(out[12345]) and not out[:12345].any()


def test_equal_calls_give_equal_bits():
    dev = [torch.randn(300000, device=DEV), torch.randn(1234567, device=DEV).to(BF16)]
    outs = [[torch.empty_like(d) for d in dev] for _ in range(2)]
    norms = [L.clip_grad_norm(dev, 1.0, out=o) for o in outs]
    torch.cuda.synchronize()
    assert torch.equal(*norms) and all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("in_place", [True, False])
def test_beyond_the_cooperative_threshold_and_31_bits(in_place):
    """One tensor of more than 2^31 elements beside a small one (the norm by
    64-bit sums of slices; results compared on slices at both ends)."""
    n = (1 << 31) + 12345
    big = torch.full((n,), 1.0 / 1024, dtype=BF16, device=DEV)
    small = torch.randn(1000, generator=torch.Generator().manual_seed(3)).to(F32)
    big[::4097] = 0.5
    dev = small.to(DEV)
    total = float(small.double().square().sum())
    for i in range(0, n, 1 << 28):
        total += float(big[i:i + (1 << 28)].double().square().sum())
    ref = math.sqrt(total)
    ends = [big[:5000].cpu(), big[-5000:].cpu(), small]
    out = None if in_place else [torch.empty_like(big), torch.empty_like(dev)]
    norm = L.clip_grad_norm([big, dev], 1.0, out=out)
    torch.cuda.synchronize()
    assert abs(float(norm) - ref) <= 2.0 ** -18 * ref
    rb, rs = (big, dev) if in_place else out
    for src, got in zip(ends, (rb[:5000], rb[-5000:], rs)):
        want = src.double() / (ref + 1e-6)
        R.check(got, want, (2.0 ** -18 + 2.0 ** -23) * want.abs(), "ends")

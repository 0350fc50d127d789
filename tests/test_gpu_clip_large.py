"""The clip on lists beyond the cooperative launch's threshold (80 MB) and on
lists of 65 to 512 tensors, every element compared on the device.

Bounds as in test_gpu_clip: squares are summed in FP32 over at most 33 elements
and in FP64 beyond, so the norm is within 2^-18 of the 64-bit one; a result is
within that, the scale's own rounding (2^-23) and one rounding of its dtype.
"""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
P = {F16: 11, BF16: 8, F32: 24}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}

LISTS = {
    # beyond 80 MB: a few tensors, and a hundred that start at any element
    "few": [(30_000_001, BF16), (9_999_999, F32), (20_000_003, F16)],
    "hundred": [(300_007 + 4099 * i, (F16, BF16, F32)[i % 3]) for i in range(100)],
    # two launches, 65 to 512 tensors
    "short65": [(7 + 331 * (i % 50), (F16, BF16, F32)[i % 3]) for i in range(65)],
    "short512": [(1 + 97 * (i % 400), (F32, F16, BF16)[i % 3]) for i in range(512)],
}


def _tensors(name):
    """Views of one buffer per dtype, each starting an odd number of elements
    after the last one's end, and the buffers."""
    g = torch.Generator(device=DEV).manual_seed(len(name))
    sizes = LISTS[name]
    flat = {dt: torch.empty(sum(n + 3 for n, t in sizes if t == dt) + 1, dtype=dt, device=DEV) for dt in P}
    at, out = dict.fromkeys(flat, 1), []
    for i, (n, dt) in enumerate(sizes):
        v = flat[dt][at[dt]:at[dt] + n]
        v.copy_(torch.randn(n, generator=g, device=DEV).mul_(0.01 * (1 + i % 7)))
        out.append(v)
        at[dt] += n + 1 + 2 * (i % 2)
    return out, flat


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("above", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
def test_every_element(name, above, in_place):
    src, flat = _tensors(name)
    kept = [t.clone() for t in src]
    guard = {dt: f.clone() for dt, f in flat.items()}
    norm64 = float(torch.stack([t.double().square().sum() for t in kept]).sum().sqrt())
    max_norm = norm64 * (2.0 if above else 0.3)
    out = None if in_place else [torch.full_like(t, float("nan")) for t in src]
    norm = L.clip_grad_norm(src, max_norm, out=out)
    torch.cuda.synchronize()
    assert abs(float(norm) - norm64) <= 2.0 ** -18 * norm64
    scale = min(1.0, max_norm / (norm64 + 1e-6))
    for i, (k, got) in enumerate(zip(kept, src if in_place else out)):
        want = k.double() * scale
        if above:
            assert torch.equal(got, k), i
            continue
        lim = (2.0 ** -18 + 2.0 ** -23) * want.abs()
        lim += 2.0 ** -P[k.dtype] * (want.abs() + lim) + TINY[k.dtype]
        assert bool(((got.double() - want).abs() <= lim).all()), i
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(src, kept))
    # nothing between or around the tensors was written
    for t, k in zip(src, kept):
        t.copy_(k)
    assert all(torch.equal(f.view(torch.int16 if f.element_size() == 2 else torch.int32),
                           guard[dt].view(torch.int16 if f.element_size() == 2 else torch.int32))
               for dt, f in flat.items())


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_an_infinite_max_norm(dt):
    """Never clips a finite norm; an infinite one over it is NaN, as in the formula."""
    t = torch.linspace(-3, 3, 20001).to(dt).to(DEV)
    kept = t.clone()
    norm = float(L.clip_grad_norm([t], float("inf")))
    ref = float(kept.double().norm())
    assert torch.equal(t, kept) and abs(norm - ref) <= 2.0 ** -18 * ref
    t[7] = float("inf")
    assert float(L.clip_grad_norm([t], float("inf"))) == float("inf") and torch.isnan(t).all()

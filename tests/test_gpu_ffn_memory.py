"""The feed-forward calls where device memory is short: sums that were to be
split over K go unsplit; a workspace that torch's cache holds the memory of is
taken from it."""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16 = torch.float16


def _fill():
    """Tensors that leave less than 2 MB of the device's memory."""
    torch.cuda.empty_cache()
    held, size = [], torch.cuda.mem_get_info()[0]
    while size >= 1 << 20:
        try:
            held.append(torch.empty(size, dtype=torch.uint8, device=DEV))
        except torch.cuda.OutOfMemoryError:
            size = (size // 2) >> 20 << 20
    return held


def _ints(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-2, 3, s, generator=g).to(F16).to(DEV) for s in shapes]


def test_split_sums_without_a_workspace():
    """64 x 1024 x 8192 splits K on the forward call and on dx: 4 MB of partial
    sums and more.  Results are sums of integers, the same either way."""
    M, N, K = 64, 1024, 8192
    x, wg, wu = _ints(1, (M, K), (N, K), (N, K))
    dy, xb, w = _ints(2, (M, K), (M, N), (K, N))      # gradients of a [K, N] weight: dx sums over K
    h, g, u = L.gated_linear(x, wg, wu, save=True)     # (the kernels are loaded)
    want = L.linear_backward(dy, xb, w, need_db=False)
    s = torch.cuda.Stream()
    out = [torch.empty(M, N, dtype=F16, device=DEV) for _ in range(3)]
    dx, dw = torch.empty(M, N, dtype=F16, device=DEV), torch.empty(K, N, dtype=F16, device=DEV)
    torch.cuda.synchronize()
    held = _fill()
    try:
        assert torch.cuda.mem_get_info()[0] < 4 << 20
        rc = [L.poot_gated_linear(L.GatedLinearArgs(
            x=x.data_ptr(), wg=wg.data_ptr(), wu=wu.data_ptr(), h=out[0].data_ptr(), g=out[1].data_ptr(),
            u=out[2].data_ptr(), M=M, N=N, K=K), s.cuda_stream),
            L.poot_linear_backward(L.LinearBackwardArgs(
                dy=dy.data_ptr(), x=xb.data_ptr(), w=w.data_ptr(), dx=dx.data_ptr(), dw=dw.data_ptr(), M=M, N=K, K=N),
                s.cuda_stream)]
        s.synchronize()
    finally:
        held.clear()
        torch.cuda.empty_cache()
    assert rc == [L.POOT_OK, L.POOT_OK]
    assert L.poot_linear_device_status(0) == L.POOT_OK
    assert torch.equal(out[1], g) and torch.equal(out[2], u)
    assert torch.equal(out[0], h)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_a_workspace_that_torch_holds_the_memory_of():
    """dg and du (4.3 GB) where 2 GB are free and torch's cache holds the rest unused."""
    M, N = 65536, 16384
    t = torch.ones(M, N, dtype=F16, device=DEV)
    x, w = torch.ones(M, 8, dtype=F16, device=DEV), torch.ones(N, 8, dtype=F16, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.empty(torch.cuda.mem_get_info()[0] - (2 << 30), dtype=torch.uint8, device=DEV)
    del held
    assert torch.cuda.mem_get_info()[0] < 3 << 30
    with torch.cuda.stream(s):
        out = L.gated_linear_backward(t, x, w, w, t, t, need_dx=False, need_dw=False, need_db=True)
    s.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    # silu(1) = 0.7311, silu'(1) = 0.9277: 65536 equal terms, one rounding
    for got, v in zip(out[3:], (0.92767051187, 0.73105857863)):
        assert bool(((got.double() / (M * v) - 1).abs() <= 2.0 ** -11 + 2.0 ** -18).all())

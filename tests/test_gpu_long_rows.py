"""The linear over rows of nearly 2^31 elements (exact: small integers at a few
places, zeros elsewhere).  In 32 bits, K rounded up to the warps' slices and the
last staged chunk's end pass 2^31."""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,variant", [(1, (1 << 31) - 8, "gemv"), (3, (1 << 31) - 8, "gemv"),
                                         (9, (1 << 31) - 8, "gemv"), (1, (1 << 31) - 1, "gemv_scalar")])
def test_rows_up_to_31_bits(M, K, variant):
    dev = "cuda:0"
    at = [0, 9, K // 16 * 7 + 5, K // 2, K // 16 * 15 + 3, K - 513, K - 2, K - 1]
    x = torch.zeros(M, K, dtype=torch.float16, device=dev)
    w = torch.zeros(1, K, dtype=torch.float16, device=dev)
    b = torch.ones(1, dtype=torch.float16, device=dev)
    for i, k in enumerate(at):
        w[0, k] = i + 1
        for m in range(M):
            x[m, k] = (i + m) % 5 - 1
    y = L.linear(x, w, b)
    torch.cuda.synchronize()
    assert L.VARIANT_NAMES[L.variant_for(x, w, b, y)] == variant
    assert L.poot_linear_device_status(0) == L.POOT_OK
    assert y[:, 0].tolist() == [float(1 + sum((i + 1) * ((i + m) % 5 - 1) for i in range(len(at)))) for m in range(M)]


def test_a_product_behind_a_kernel_of_seconds():
    """The GEMM's bounded waits (two seconds) start when the previous kernel in
    the stream has ended, although its blocks may be resident before: here
    behind a single block's pass over 2^31 - 1 elements."""
    dev, K = "cuda:0", (1 << 31) - 1
    x = torch.zeros(1, K, dtype=torch.float16, device=dev)
    w = torch.zeros(1, K, dtype=torch.float16, device=dev)
    b = torch.ones(1, dtype=torch.float16, device=dev)
    g = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).half()
    dy, xs, ws = ints(300, 264), ints(300, 200), ints(264, 200)
    dev_in = [t.to(dev) for t in (dy, xs, ws)]
    L.linear_backward(*dev_in)   # (the workspace and the kernels are there)
    torch.cuda.synchronize()
    y = torch.empty(1, 1, dtype=torch.float16, device=dev)
    L.linear(x, w, b, out=y)
    dx, dw, db = L.linear_backward(*dev_in)
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    d = dy.double()
    assert (y == 1).all()
    for o, r in ((dx, d @ ws.double()), (dw, d.T @ xs.double()), (db, d.sum(0))):
        assert torch.equal(o.cpu(), r.half())

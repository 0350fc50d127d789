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

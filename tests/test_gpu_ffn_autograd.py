"""The feed-forward calls beside torch's automatic differentiation: results carry
no graph, and tensors written to count as modified."""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _t(*shape):
    return torch.ones(shape, dtype=torch.float16, device=DEV)


def test_results_carry_no_graph():
    x, w = _t(20, 16).requires_grad_(), _t(24, 16).requires_grad_()
    h, g, u = L.gated_linear(x, w, w, save=True)
    grads = L.gated_linear_backward(h, x, w, w, g, u, need_db=True)
    assert not any(t.requires_grad for t in (h, g, u, *grads))


@pytest.mark.parametrize("write", ["in place", "out", "gated out"])
def test_a_graph_notices_that_a_tensor_it_saved_was_written(write):
    saved = _t(24, 24)
    w = _t(24, 24).requires_grad_()
    y = (w * saved).sum()
    before = saved._version
    if write == "in place":
        L.clip_grad_norm([_t(5), saved], 0.5)
    elif write == "out":
        L.clip_grad_norm([_t(24, 24)], 0.5, out=[saved])
    else:
        L.gated_linear(_t(24, 8), _t(24, 8), _t(24, 8), out=saved)
    assert saved._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inputs_that_are_only_read_keep_their_version():
    src, out = _t(100), _t(100)
    before = src._version
    L.clip_grad_norm([src], 0.5, out=[out])
    assert src._version == before


def test_tensors_made_in_inference_mode():
    with torch.inference_mode():
        t = _t(100)
        norm = L.clip_grad_norm([t], 0.5)
    norm = L.clip_grad_norm([t], 0.25)
    assert abs(float(norm) - 0.5) < 2.0 ** -9

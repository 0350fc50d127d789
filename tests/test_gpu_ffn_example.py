"""The feed-forward operators together: the training example, and one step's
gradients against automatic differentiation of the same block in FP32."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_gated_ffn.py")


def _example():
    spec = importlib.util.spec_from_file_location("train_gated_ffn", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_learns_and_decodes():
    ex = _example()
    losses, norms, block = ex.train(steps=30, rows=512)
    assert all(n > 0 for n in norms)
    assert losses[-1] < 0.7 * losses[0], losses
    # y is of order 1 and rounded to bfloat16 on both ways, h before it: a
    # few steps of 2^-8 of the largest |y| (about 4)
    assert ex.decode(block) <= 4 * 2.0 ** -8 * 4


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh", "gelu_erf"])
def test_one_step_against_automatic_differentiation(activation):
    ex = _example()
    block = ex.Block(128, 320, 5, activation=activation)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(300, 128, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(300, 128, generator=gen, device="cuda").bfloat16()
    _, saved = block.forward(x, save=True)
    grads = block.gradients(x, saved, dy)
    ws = [w.float().requires_grad_() for w in (block.wg, block.wu, block.wd)]
    act = {"silu": torch.nn.functional.silu,
           "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
           "gelu_erf": torch.nn.functional.gelu}[activation]
    ((act(x.float() @ ws[0].T) * (x.float() @ ws[1].T)) @ ws[2].T).backward(dy.float())
    # roundings to bfloat16 on the way (h, g, u, dh, dg or du, the result), each
    # about 0.42 2^-8 rms of a value: 2^-7 bounds their root mean square
    for got, w in zip(grads, ws):
        assert float((got.float() - w.grad).norm() / w.grad.norm()) <= 2.0 ** -7

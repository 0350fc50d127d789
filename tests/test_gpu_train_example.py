"""The training operators together: the next-token example runs with either kind
of state, and one step's gradients against automatic differentiation in FP32."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_next_token.py")


def _example():
    spec = importlib.util.spec_from_file_location("train_next_token", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_runs(bits):
    ex = _example()
    losses, norms, model = ex.train(steps=4, rows=300, vocab=501, dim=72, hidden=96, bits=bits)
    assert all(math.isfinite(v) for v in losses) and all(n > 0 for n in norms)
    assert model.steps == 4
    for m, w in zip(model.masters, model.weights):
        assert torch.equal(m.bfloat16(), w)
    tokens = torch.randint(0, 501, (7,), device="cuda")
    assert bool(model.forward(tokens, tokens).isfinite().all())


def test_one_step_against_automatic_differentiation():
    ex = _example()
    model = ex.Model(701, 96, 128, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randint(0, 701, (701, 4), generator=gen, device="cuda")
    tokens, targets = ex.text(333, 701, gen, table)
    _, saved = model.forward(tokens, targets, save=True)
    grads = model.gradients(tokens, targets, saved)
    emb, wg, wu, wd, head = ws = [w.float().requires_grad_() for w in model.weights]
    x = emb[tokens]
    y = (torch.nn.functional.silu(x @ wg.T) * (x @ wu.T)) @ wd.T + x
    torch.nn.functional.cross_entropy(y @ head.T, targets, ignore_index=ex.IGNORE).backward()
    # roundings to bfloat16 on the way (h, y twice, q, dy, dh, dg or du, dx, the result), each
    # about 0.42 2^-8 rms of a value: 2^-7 bounds the root of the sum of nine squares, 1.26 2^-8
    for got, w in zip(grads, ws):
        assert float((got.float() - w.grad).norm() / w.grad.norm()) <= 2.0 ** -7

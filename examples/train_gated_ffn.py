"""Train a gated feed-forward block on synthetic data, then decode with it.

    python examples/train_gated_ffn.py [--steps 30] [--rows 2048]

One step, as a training program runs it:

    h, g, u = gated_linear(x, wg, wu, save=True)      act(x Wg^T) * (x Wu^T)
    y       = contract(h, wd)                         the down projection
    dh, dwd = linear_backward(dy, h, wd)
    dwg, dwu = gated_linear_backward(dh, x, wg, wu, g, u)
    norm    = clip_grad_norm([dwg, dwu, dwd], max_norm)
    weights -= rate * gradients                       FP32 masters, bfloat16 copies

The target is another block of the same shape with fixed random weights.
Decoding runs single rows through the same calls (M = 1: the GEMV kernels).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_fp16_gb300 as L  # noqa: E402


class Block:
    """FP32 master weights of a gated block and their bfloat16 copies."""

    def __init__(self, dim: int, hidden: int, seed: int, device="cuda", activation: str = "silu"):
        gen = torch.Generator().manual_seed(seed)
        self.activation = activation
        self.masters = [(torch.randn(s, generator=gen) * (s[1] ** -0.5)).to(device)
                        for s in ((hidden, dim), (hidden, dim), (dim, hidden))]
        self.refresh()

    def refresh(self):
        self.wg, self.wu, self.wd = (m.bfloat16() for m in self.masters)

    def forward(self, x, save: bool = False):
        out = L.gated_linear(x, self.wg, self.wu, activation=self.activation, save=save)
        h = out[0] if save else out
        y = L.contract(h, self.wd)
        return (y, out) if save else y

    def gradients(self, x, saved, dy):
        h, g, u = saved
        dh, dwd, _ = L.linear_backward(dy, h, self.wd, need_db=False)
        _, dwg, dwu, _, _ = L.gated_linear_backward(dh, x, self.wg, self.wu, g, u, activation=self.activation,
                                                    need_dx=False)
        return [dwg, dwu, dwd]

    def update(self, grads, rate: float):
        for m, d in zip(self.masters, grads):
            m.add_(d.float(), alpha=-rate)
        self.refresh()


def train(steps: int = 30, rows: int = 2048, dim: int = 256, hidden: int = 1024, rate: float = 0.5,
          max_norm: float = 1.0, log=None):
    """Losses and gradient norms of the steps, and the trained block."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    teacher, block = Block(dim, hidden, 2), Block(dim, hidden, 3)
    losses, norms = [], []
    for step in range(steps):
        x = torch.randn(rows, dim, generator=gen, device="cuda").bfloat16()
        target = teacher.forward(x).float()
        y, saved = block.forward(x, save=True)
        diff = y.float() - target
        losses.append(diff.square().mean())
        dy = (diff * (2.0 / dim)).bfloat16()  # rows' gradients; the mean over rows goes into the rate
        grads = block.gradients(x, saved, dy)
        norms.append(L.clip_grad_norm(grads, max_norm))
        block.update(grads, rate)
        if log and (step % 5 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {float(losses[-1]):.4f}  gradient norm {float(norms[-1]):.2f}")
    return [float(v) for v in losses], [float(v) for v in norms], block


def decode(block: Block, tokens: int = 4, dim: int = 256):
    """Largest difference between rows decoded one by one and the batch."""
    x = torch.randn(tokens, dim, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    one_by_one = torch.cat([block.forward(x[i:i + 1]) for i in range(tokens)])
    return float((one_by_one.float() - block.forward(x).float()).abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--rows", type=int, default=2048)
    a = ap.parse_args()
    losses, _, block = train(a.steps, a.rows, log=print)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    print(f"single rows against the batch: largest difference {decode(block):.4g}")


if __name__ == "__main__":
    main()

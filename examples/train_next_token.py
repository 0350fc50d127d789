"""Train a small next-token model on synthetic text, from the loss to the update.

    python examples/train_next_token.py [--steps 40] [--rows 2048] [--bits 8]

One step, as a training program runs it:

    x        = embedding[tokens]
    h, g, u  = gated_linear(x, wg, wu, save=True)          act(x Wg^T) * (x Wu^T)
    y        = contract(h, wd, steps=[("add", x)])         the down projection, residual
    loss, lse = linear_cross_entropy(y, head, targets, save=True)
    dy, dhead = linear_cross_entropy_backward(dloss, y, head, targets, lse)
    dh, dwd   = linear_backward(dy, h, wd)
    dx, dwg, dwu = gated_linear_backward(dh, x, wg, wu, g, u)
    norm      = clip_grad_norm(gradients, max_norm)
    adamw_step(masters, gradients, state, copies=weights)  FP32 masters, bfloat16 copies

The text is drawn from a fixed random table of next tokens; a few targets are
left out of the loss (the ignored index), as padding is.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_fp16_gb300 as L  # noqa: E402

IGNORE = -100


class Model:
    """FP32 master weights, their bfloat16 copies and the AdamW state."""

    def __init__(self, vocab: int, dim: int, hidden: int, seed: int = 3, bits: int = 32, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        shapes = ((vocab, dim), (hidden, dim), (hidden, dim), (dim, hidden), (vocab, dim))
        self.masters = [(torch.randn(s, generator=gen) * (s[1] ** -0.5)).to(device) for s in shapes]
        self.weights = [m.bfloat16() for m in self.masters]
        self.state = L.adamw_state(self.masters, bits=bits)
        self.steps = 0

    def forward(self, tokens, targets, save: bool = False):
        """The rows' losses; with `save` also what `gradients` reads."""
        emb, wg, wu, wd, head = self.weights
        x = emb[tokens]
        h, g, u = L.gated_linear(x, wg, wu, save=True)
        y = L.contract(h, wd, steps=[("add", x)])
        if not save:
            return L.linear_cross_entropy(y, head, targets, ignore_index=IGNORE)
        loss, lse = L.linear_cross_entropy(y, head, targets, ignore_index=IGNORE, save=True)
        return loss, (x, h, g, u, y, lse)

    def gradients(self, tokens, targets, saved):
        """Gradients of the mean loss over the targets in use, in the order of the weights."""
        emb, wg, wu, wd, head = self.weights
        x, h, g, u, y, lse = saved
        dloss = (1.0 / (targets != IGNORE).sum().clamp(min=1)).float().expand(len(targets))
        dy, dhead, _ = L.linear_cross_entropy_backward(dloss, y, head, targets, lse, ignore_index=IGNORE)
        dh, dwd, _ = L.linear_backward(dy, h, wd, need_db=False)
        dx, dwg, dwu, _, _ = L.gated_linear_backward(dh, x, wg, wu, g, u)
        demb = torch.zeros(emb.shape, device=emb.device).index_add_(0, tokens, dx.float() + dy.float())
        return [demb, dwg, dwu, dwd, dhead]

    def update(self, grads, rate: float, max_norm: float = 1.0):
        norm = L.clip_grad_norm(grads, max_norm)
        self.steps += 1
        L.adamw_step(self.masters, grads, self.state, step=self.steps, lr=rate, copies=self.weights)
        return norm


def text(rows: int, vocab: int, gen, table):
    """Tokens and what follows them; one in sixteen targets is padding."""
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    follow = table[tokens, torch.randint(0, table.shape[1], (rows,), generator=gen, device="cuda")]
    pad = torch.rand(rows, generator=gen, device="cuda") < 1 / 16
    return tokens, torch.where(pad, IGNORE, follow)


def train(steps: int = 40, rows: int = 2048, vocab: int = 2000, dim: int = 128, hidden: int = 256, rate: float = 3e-3,
          bits: int = 32, log=None):
    """Mean losses and gradient norms of the steps, and the trained model."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randint(0, vocab, (vocab, 4), generator=gen, device="cuda")
    model = Model(vocab, dim, hidden, bits=bits)
    losses, norms = [], []
    for step in range(steps):
        tokens, targets = text(rows, vocab, gen, table)
        loss, saved = model.forward(tokens, targets, save=True)
        losses.append(loss.sum() / (targets != IGNORE).sum())
        norms.append(model.update(model.gradients(tokens, targets, saved), rate))
        if log and (step % 5 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {float(losses[-1]):.4f}  gradient norm {float(norms[-1]):.3f}")
    return [float(v) for v in losses], [float(v) for v in norms], model


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--bits", type=int, default=32, choices=(32, 8))
    a = ap.parse_args()
    losses, _, _ = train(a.steps, a.rows, bits=a.bits, log=print)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()

"""Plain 64-bit forms of the vocabulary head's loss and gradients, and their bounds.

Elementwise bounds, from the operators' stated numerics (u = 2^-24):
* a logit: FP32 sums of K products.  The tensor core adds 16 products to the
  running sum with one truncation of at most 2^-23 of the larger side.  The loss
  sums chunks of 1024 that way and rounds K / 1024 additions to nearest; the
  gradients sum up to 32768 (ffn_ref.acc_err);
* exp(z - m): the exponent z log2(e) - m log2(e) in one fused operation, off by
  2^-24 of |z| log2(e) twice (constant and rounding), ex2 by 2^-22 of the result:
  relative 2^-21 + |z| 2^-22 in all; results below 2^-126 are dropped, in the
  gradients after a factor of 2^14: probabilities below 2^-140;
* a row's sum of V exponentials: at most 64 rounded additions one after the other
  at the sizes tested;
* q is rounded to the head dtype (p = 11 or 8 bits) times a power of two that
  puts the largest |dloss| at 2^14 or above: u_p of itself, and in binary16 a step of 2^-25
  over that power;
* a column's sum for db is one of unrounded values;
* results are rounded once.
"""
import torch

from .ffn_ref import P, TINY, acc_err

IGNORE = -100


def head_acc(K):
    return (min(K, 1024) / 16 + 64) * 2.0 ** -23 + (K / 1024) * 2.0 ** -24


def logits64(x, w, b, acc):
    x, w = x.double(), w.double()
    z, e = x @ w.T, acc * (x.abs() @ w.abs().T)
    if b is not None:
        z, e = z + b.double(), e + b.double().nan_to_num(posinf=0, neginf=0).abs() * 2.0 ** -23
    return z, e


def loss64(x, w, target, b, ignore=IGNORE):
    """(loss, its bound, lse, its bound); finite logits."""
    z, ez = logits64(x, w, b, head_acc(x.shape[1]))
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    big = z.nan_to_num(neginf=0).abs().amax(1)
    el = ((p * ez).sum(1) + ez.nan_to_num().amax(1) * 2.0 ** -10  # (second order)
          + 2.0 ** -21 + big * 2.0 ** -22 + 64 * 2.0 ** -24 + lse.abs() * 2.0 ** -23)
    used = target != ignore
    t = torch.where(used, target, 0)[:, None]
    loss = torch.where(used, lse - z.gather(1, t)[:, 0], 0.0)
    bound = torch.where(used, el + ez.gather(1, t)[:, 0] + loss.abs() * 2.0 ** -23, 0.0)
    return loss, bound, lse, el


def grads64(dloss, x, w, target, lse, b, ignore=IGNORE):
    """[(dx, bound), (dw, bound), (db, bound)] before the last rounding."""
    dt = x.dtype
    used = target != ignore
    x = torch.where(used[:, None], x, 0)  # (what ignored rows hold plays no part)
    M, K = x.shape
    V = w.shape[0]
    z, ez = logits64(x, w, b, acc_err(K))
    lse = torch.where(used, lse, 0.0).double()[:, None]
    p = torch.where(used[:, None], torch.exp(z - lse), 0.0)
    ep = p * torch.expm1(ez + 2.0 ** -21 + (z.abs() + lse.abs()).nan_to_num(posinf=0) * 2.0 ** -22) + 2.0 ** -140
    d = torch.where(used, dloss, 0.0).double()[:, None]
    q = p.scatter_add(1, torch.where(used, target, 0)[:, None], -used.double()[:, None]) * d
    eq = d.abs() * ep + q.abs() * 2.0 ** -22
    ef = eq  # before it is rounded
    tiny = TINY[dt] * float(d.abs().max()) * 2.0 ** -14
    eq = eq + (q.abs() + eq) * 2.0 ** -P[dt] + tiny
    qa = q.abs() + eq
    X, W = x.double(), w.double()
    return [(q @ W, eq @ W.abs() + acc_err(V) * (qa @ W.abs())),
            (q.T @ X, eq.T @ X.abs() + acc_err(M) * (qa.T @ X.abs())),
            (q.sum(0), ef.sum(0) + (M / 8 + 64) * 2.0 ** -24 * qa.sum(0))]


def check(got, ref, err, name):
    """got (float32, or rounded once to its dtype) against ref known to err."""
    g = got.double()
    lim = err if got.dtype == torch.float32 else err + (ref.abs() + err) * 2.0 ** -P[got.dtype] + TINY[got.dtype]
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    bad = ~((g - ref).abs() <= lim)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((g - ref).abs() / lim).nan_to_num(posinf=9e9).max()):.3g} times it")

"""Plain 64-bit forms of the feed-forward operators and their error bounds.

Bounds, elementwise, derived from the operators' stated numerics (p = 11 for
binary16, 8 for bfloat16; u_p = 2^-p, half the spacing relative to a value):
* a sum of L products in FP32: |error| <= ACC(L) * sum |terms|, ACC(L) =
  (L / 16 + 64) 2^-23: the tensor core adds 16 products (exact) to the running
  sum with one truncation of at most 2^-23 of the larger side, the GEMVs and
  split sums round fewer times than that;
* an activation in FP32: relative error at most 2^-18 of |t| (exponential and
  division to a few ulps, the exponent's argument amplified by |t| <= 90), and
  a Lipschitz constant of 1.13 (the GELUs' largest slope), 1.1 for silu;
* dg and du are rounded to the head dtype before the products: each term of
  dx and dW moves by at most u_p of itself, plus the format's smallest step;
* the result is rounded once: u_p |value| plus the format's smallest step.
"""
import math

import torch

P = {torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
LIP = 1.13
ACT_ERR = 2.0 ** -18


def acc_err(length):
    return (length / 16 + 64) * 2.0 ** -23


def act64(name, t):
    if name == "silu":
        return t / (1 + torch.exp(-t))
    if name == "gelu_tanh":
        return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    return 0.5 * t * (1 + torch.erf(t / math.sqrt(2)))


def act_grad64(name, t):
    """By automatic differentiation of the value, in 64 bits."""
    v = t.detach().clone().requires_grad_(True)
    act64(name, v).sum().backward()
    return v.grad


def rounded(err, ref, dt):
    """Bound after rounding ref (known to err) once to dt."""
    return err + (ref.abs() + err) * 2.0 ** -P[dt] + TINY[dt]


def gated64(x, wg, wu, bg, bu, act):
    """(h, g, u) and their bounds before rounding."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    N, K = wg.shape
    zero = torch.zeros(N, dtype=torch.float64)
    bg = zero if bg is None else bg.double()
    bu = zero if bu is None else bu.double()
    g, u = x @ wg.T + bg, x @ wu.T + bu
    eg = acc_err(K) * (x.abs() @ wg.abs().T + bg.abs())
    eu = acc_err(K) * (x.abs() @ wu.abs().T + bu.abs())
    a = act64(act, g)
    ea = LIP * eg + ACT_ERR * g.abs()
    return (a * u, g, u), (ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -22 * (a * u).abs(), eg, eu)


def gate_grad64(dh, g, u, act):
    dh, g, u = dh.double(), g.double(), u.double()
    dg, du = dh * u * act_grad64(act, g), dh * act64(act, g)
    # the derivative's own error: its terms reach |t| of magnitude in (1 + |t|)
    eg = ACT_ERR * dh.abs() * u.abs() * (1 + g.abs())
    eu = ACT_ERR * dh.abs() * g.abs()
    return (dg, du), (eg, eu)


def product_bound(a, ea, b, dt_round):
    """Bound of sum_k a b over a's last and b's first dim; a known to ea, then
    (with dt_round) rounded to that dtype before the product."""
    if dt_round is not None:
        ea = rounded(ea, a, dt_round)
    return ea @ b.abs() + acc_err(a.shape[-1]) * ((a.abs() + ea) @ b.abs())


def check(got, ref, err, name):
    """got (rounded once to its dtype) against ref known to err."""
    dt = got.dtype
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    diff = (got.detach().cpu().double() - ref).abs()
    lim = rounded(err, ref, dt)
    bad = ~(diff <= lim)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float((diff / lim).nan_to_num(posinf=9e9).max()):.3g} times it")


def rms(got, ref, name, limit):
    """Relative root-mean-square error: roundings are independent, so far
    below the elementwise worst case."""
    d = (got.detach().cpu().double() - ref)
    r = float(d.norm() / ref.norm().clamp_min(1e-300))
    assert r <= limit, f"{name}: relative rms error {r:.3g} > {limit:.3g}"

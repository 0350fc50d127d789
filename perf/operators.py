"""The feed-forward operators as they are measured: cases, plain forms, calls.

    gated     h = act(x Wg^T + bg) * (x Wu^T + bu), x [M, K], Wg and Wu [N, K]
              (with `save`, g and u rounded to the head dtype as well)
    gated_bwd its gradients: dg = dh * u * act'(g), du = dh * act(g),
              dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dbg, dbu
    linear_bwd the gradients of y = x W^T + b: dx = dy W, dW = dy^T x, db
    clip      the norm over a list of gradient tensors, and the tensors
              scaled by min(1, max_norm / (norm + 1e-6))

`run` computes an operator in elementary torch operations in 32 bits, rounded
once at the end, or, with `own` set, through the framework's entry points.
Sizes are those of the framework's workloads (the toy linear, the ragged
shape, decode rows, the 4096 prefill projection, the MLP projection).
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_ACTS = ("silu", "gelu_tanh", "gelu_erf")
_DEV = "cuda"
_EPS = 1e-6  # added to the norm before the division


def listed():
    return [
        # one token through the MLP of a decode step: both weights are
        # streamed once, the two products share the one row of x
        dict(name="gated_decode_m1", op="gated", M=1, N=14336, K=4096, dtype="bf16", act="silu", bias=False,
             save=False),
        # a small decode batch on a small block, the shortest useful call
        dict(name="gated_decode_m8", op="gated", M=8, N=4096, K=4096, dtype="f16", act="gelu_tanh", bias=True,
             save=False),
        # odd sizes in all three dimensions: rows that no 16-byte load fits
        dict(name="gated_ragged", op="gated", M=2047, N=1000, K=770, dtype="f16", act="gelu_erf", bias=True,
             save=True),
        # prompt processing: no state is kept for a backward pass
        dict(name="gated_prefill", op="gated", M=4096, N=4096, K=4096, dtype="f16", act="gelu_tanh", bias=False,
             save=False),
        # the forward half of a training step on the MLP projection
        dict(name="gated_train", op="gated", M=8192, N=14336, K=4096, dtype="bf16", act="silu", bias=False,
             save=True),
        # the backward half of the same step: four products' worth of work
        dict(name="gated_bwd_train", op="gated_bwd", M=8192, N=14336, K=4096, dtype="bf16", act="silu", bias=False),
        # a small model's step: one wave of tiles, launches count
        dict(name="gated_bwd_toy", op="gated_bwd", M=1024, N=1024, K=768, dtype="f16", act="gelu_tanh", bias=True),
        # odd sizes, biases, a short batch
        dict(name="gated_bwd_ragged", op="gated_bwd", M=333, N=1000, K=770, dtype="bf16", act="gelu_erf", bias=True),
        # the down projection's gradients in the same step
        dict(name="linear_bwd_down", op="linear_bwd", M=8192, N=4096, K=14336, dtype="bf16", bias=False),
        # the toy linear's gradients
        dict(name="linear_bwd_toy", op="linear_bwd", M=1024, N=1024, K=768, dtype="f16", bias=True),
        # all gradients of a small model, binary16, from one flat bucket:
        # tensors start at any element
        dict(name="clip_small", op="clip", layers=2, N=1000, K=770, dtype="f16", flat=True, max_norm=1.0),
        # weight gradients of four blocks in bfloat16, their biases in FP32
        dict(name="clip_blocks", op="clip", layers=4, N=14336, K=4096, dtype="mixed", flat=False, max_norm=1.0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Log-uniform; a third are multiples of 64, a third of 8, a third any."""
    v = _logint(rng, lo, hi)
    step = rng.choice((64, 8, 1))
    return max(lo, min(hi, v // step * step or step))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_bwd", "linear_bwd", "clip"))
    if op == "clip":
        return dict(op=op, layers=rng.randint(1, 4), N=_size(rng, 64, 14336), K=_size(rng, 64, 4096),
                    dtype=rng.choice(("f16", "bf16", "f32", "mixed")), flat=rng.random() < 0.5,
                    max_norm=rng.choice((0.1, 1.0, 1e4)))
    # a third decode-sized batches, the rest up to the training step's rows
    M = _logint(rng, 1, 16) if rng.random() < 0.34 else _size(rng, 17, 8192)
    if op == "linear_bwd":
        N, K = _size(rng, 64, 4096), _size(rng, 64, 14336)
    else:
        N, K = _size(rng, 64, 14336), _size(rng, 64, 4096)
    case = dict(op=op, M=M, N=N, K=K, dtype=rng.choice(("f16", "bf16")), bias=rng.random() < 0.5)
    if op != "linear_bwd":
        case["act"] = rng.choice(_ACTS)
    if op == "gated":
        case["save"] = rng.random() < 0.5
    return case


def _clip_shapes(case):
    """(shape, dtype) of every gradient tensor: three weights and biases a layer."""
    wt = _DT["bf16" if case["dtype"] == "mixed" else case["dtype"]]
    bt = _DT["f32" if case["dtype"] == "mixed" else case["dtype"]]
    N, K = case["N"], case["K"]
    layer = [((N, K), wt), ((N, K), wt), ((K, N), wt), ((N,), bt), ((N,), bt), ((K,), bt)]
    return layer * case["layers"]


def _buckets(case):
    """Empty tensors of those shapes; with `flat`, views of one buffer per dtype."""
    shapes = _clip_shapes(case)
    if not case["flat"]:
        return [torch.empty(s, dtype=t, device=_DEV) for s, t in shapes]
    flat = {t: torch.empty(sum(math.prod(s) for s, u in shapes if u == t), dtype=t, device=_DEV)
            for t in {t for _, t in shapes}}
    at = dict.fromkeys(flat, 0)
    views = []
    for s, t in shapes:
        n = math.prod(s)
        views.append(flat[t][at[t]:at[t] + n].view(s))
        at[t] += n
    return views


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed))

    def normal(shape, std, dt):
        return (torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32) * std).to(dt)

    if case["op"] == "clip":
        grads = _buckets(case)
        for i, g in enumerate(grads):
            g.copy_(torch.randn(g.shape, generator=gen, device=_DEV, dtype=torch.float32).mul_(1e-3 * (1 + i % 5)))
        return dict(case=case, grads=grads, out=_buckets(case))
    M, N, K, dt = case["M"], case["N"], case["K"], _DT[case["dtype"]]
    st = dict(case=case, x=normal((M, K), 1.0, dt))
    if case["op"] == "linear_bwd":
        st.update(w=normal((N, K), 0.02, dt), dy=normal((M, N), 0.05, dt))
        return st
    st.update(wg=normal((N, K), 0.02, dt), wu=normal((N, K), 0.02, dt))
    if case["op"] == "gated":
        st.update(bg=normal((N,), 0.1, dt) if case["bias"] else None,
                  bu=normal((N,), 0.1, dt) if case["bias"] else None)
    else:
        std = 0.02 * math.sqrt(K)
        st.update(g=normal((M, N), std, dt), u=normal((M, N), std, dt), dh=normal((M, N), 0.05, dt))
    return st


# ---- plain forms: elementary operations in 32 bits --------------------------
def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(name, t):
    if name == "silu":
        return t * _sigmoid(t)
    if name == "gelu_tanh":
        return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))
    return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))


def _act_grad(name, t):
    if name == "silu":
        s = _sigmoid(t)
        return s * (1.0 + t * (1.0 - s))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (t + 0.044715 * t * t * t))
        return 0.5 * (1.0 + th) + 0.5 * t * (1.0 - th * th) * c * (1.0 + 3.0 * 0.044715 * t * t)
    return 0.5 * (1.0 + torch.erf(t * math.sqrt(0.5))) + t * torch.exp(-0.5 * t * t) / math.sqrt(2.0 * math.pi)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "clip":
        sums = [g.float().square().sum() for g in st["grads"]]
        norm = torch.sqrt(torch.stack(sums).sum())
        scale = torch.clamp(case["max_norm"] / (norm + _EPS), max=1.0)
        return [norm] + [(g.float() * scale).to(g.dtype) for g in st["grads"]]
    dt = _DT[case["dtype"]]
    x = st["x"].float()
    if op == "linear_bwd":
        dy = st["dy"].float()
        out = [(dy @ st["w"].float()).to(dt), (dy.T @ x).to(dt)]
        return out + ([dy.sum(0).to(dt)] if case["bias"] else [])
    wg, wu = st["wg"].float(), st["wu"].float()
    if op == "gated":
        g, u = x @ wg.T, x @ wu.T
        if case["bias"]:
            g, u = g + st["bg"].float(), u + st["bu"].float()
        h = (_act(case["act"], g) * u).to(dt)
        return [h, g.to(dt), u.to(dt)] if case["save"] else [h]
    g, u, dh = st["g"].float(), st["u"].float(), st["dh"].float()
    dg = dh * u * _act_grad(case["act"], g)
    du = dh * _act(case["act"], g)
    out = [(dg @ wg + du @ wu).to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt)]
    return out + ([dg.sum(0).to(dt), du.sum(0).to(dt)] if case["bias"] else [])


# ---- the framework's entry points -------------------------------------------
def _own(st):
    import linear_fp16_gb300 as L
    case = st["case"]
    op = case["op"]
    if op == "clip":
        norm = L.clip_grad_norm(st["grads"], case["max_norm"], out=st["out"])
        return [norm] + st["out"]
    if op == "linear_bwd":
        out = L.linear_backward(st["dy"], st["x"], st["w"], need_db=case["bias"])
    elif op == "gated":
        out = L.gated_linear(st["x"], st["wg"], st["wu"], st["bg"], st["bu"], activation=case["act"],
                             save=case["save"])
        out = out if case["save"] else (out,)
    else:
        out = L.gated_linear_backward(st["dh"], st["x"], st["wg"], st["wu"], st["g"], st["u"],
                                      activation=case["act"], need_db=case["bias"])
    return [t for t in out if t is not None]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] == "clip":
        elems = [(math.prod(s), t.itemsize) for s, t in _clip_shapes(case)]
        return {"bytes": sum(2 * n * b for n, b in elems) + 4, "flops": sum(3 * n for n, _ in elems)}
    M, N, K, b = case["M"], case["N"], case["K"], int(case["bias"])
    if case["op"] == "gated":
        outs = 3 if case["save"] else 1
        return {"bytes": 2 * (M * K + 2 * N * K + outs * M * N + 2 * b * N), "flops": 4 * M * N * K}
    if case["op"] == "linear_bwd":
        return {"bytes": 2 * (M * N + 2 * M * K + 2 * N * K + b * N), "flops": 4 * M * N * K}
    return {"bytes": 2 * (3 * M * N + 2 * M * K + 4 * N * K + 2 * b * N), "flops": 8 * M * N * K}


# ---- the definitions in 64 bits ----------------------------------------------
def _phi(act, v):
    """act(v) and act'(v) in binary64."""
    if act == "gelu_erf":
        cdf = 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        return v * cdf, cdf + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    # v sigma(z): z = v, or the tanh form's 2 sqrt(2/pi) (v + 0.044715 v^3)
    if act == "silu":
        z, dz = v, torch.ones_like(v)
    else:
        a = math.sqrt(8.0 / math.pi)
        z, dz = a * (v + 0.044715 * v.pow(3)), a * (1 + 0.134145 * v.square())
    s = torch.special.expit(z)
    return v * s, s + v * s * torch.special.expit(-z) * dz


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["grads"])
        norm = math.sqrt(total)
        factor = min(1.0, case["max_norm"] / (norm + _EPS))
        return [torch.tensor(norm, dtype=torch.float64)] + [g.double() * factor for g in st["grads"]]
    x = st["x"].double()
    if case["op"] == "linear_bwd":
        dy = st["dy"].double()
        res = [torch.mm(dy, st["w"].double()), torch.mm(dy.t(), x)]
        if case["bias"]:
            res.append(dy.sum(dim=0))
        return res
    if case["op"] == "gated":
        pre = []
        for w, b in ((st["wg"], st["bg"]), (st["wu"], st["bu"])):
            p = torch.mm(x, w.double().t())
            pre.append(p if b is None else p + b.double())
        h = _phi(case["act"], pre[0])[0] * pre[1]
        return [h] + pre if case["save"] else [h]
    a, da = _phi(case["act"], st["g"].double())
    dh = st["dh"].double()
    du = dh * a
    dg = dh * st["u"].double() * da
    del a, da, dh
    dx = torch.mm(dg, st["wg"].double())
    dx += torch.mm(du, st["wu"].double())
    res = [dx, torch.mm(dg.t(), x), torch.mm(du.t(), x)]
    if case["bias"]:
        res += [dg.sum(dim=0), du.sum(dim=0)]
    return res

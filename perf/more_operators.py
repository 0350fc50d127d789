"""The two ends of a training step as they are measured: cases, plain forms, calls.

    loss      loss_i = log sum_v exp z_iv - z_i,t(i), z = x W^T + b the logits of
              a vocabulary head, x [M, K], W [V, K], b [V]; 0 where the target
              is the ignored index (with `save`, the log-sum-exp as well)
    loss_bwd  its gradients: q = dloss_i (exp(z - lse_i) - [v = t(i)]), 0 in
              ignored rows; dx = q W, dW = q^T x, db = column sums of q
    adamw     one step over a list of tensors:
              m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
              p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
              with m and v in FP32, or in 8 bits: blocks of 256 elements with a
              scale s each, m = s c |c| for a code c of -127 .. 127, sqrt(v) =
              s c^2 for one of 0 .. 255, the codes nearest in c

`run` computes an operator in elementary torch operations in 32 bits, rounded
once at the end, or, with `own` set, through the framework's entry points.  A
step updates its tensors in place in both forms; states in 8 bits are returned
as the values they stand for.  Sizes are those of the framework's workloads (the toy linear,
the ragged shape, the 4096 prefill projection, the MLP projection's
tensors) with vocabularies of generic sizes.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"
_IGNORE = -100
_BLOCK = 256  # elements of a scale
_STEP, _LR, _B1, _B2, _EPS, _WD = 100, 1e-3, 0.9, 0.999, 1e-8, 0.1


def listed():
    return [
        # the log-probability of one token while a text is scored token by
        # token: the head's weights are streamed once
        dict(name="loss_one_token", op="loss", M=1, V=131072, K=4096, dtype="bf16", bias=False, ignore=0.0, save=False),
        # a small model's head: one wave of tiles, launches count
        dict(name="loss_toy", op="loss", M=1024, V=1024, K=768, dtype="f16", bias=True, ignore=0.0, save=True),
        # odd sizes in all three dimensions, a tenth of the rows is padding
        dict(name="loss_ragged", op="loss", M=2047, V=32003, K=770, dtype="f16", bias=True, ignore=0.1, save=False),
        # evaluation of a prompt: no state is kept for a backward pass
        dict(name="loss_prefill", op="loss", M=4096, V=65536, K=4096, dtype="f16", bias=False, ignore=0.0, save=False),
        # the forward half of a training step on a large vocabulary
        dict(name="loss_train", op="loss", M=8192, V=131072, K=4096, dtype="bf16", bias=False, ignore=0.0, save=True),
        # the small head's gradients
        dict(name="loss_bwd_toy", op="loss_bwd", M=1024, V=1024, K=768, dtype="f16", bias=True, ignore=0.0,
             weighted=False),
        # odd sizes, a short batch, weighted tokens, half of them prompt that carries no loss
        dict(name="loss_bwd_ragged", op="loss_bwd", M=333, V=32003, K=770, dtype="bf16", bias=True, ignore=0.5,
             weighted=True),
        # the backward half of the training step
        dict(name="loss_bwd_train", op="loss_bwd", M=8192, V=131072, K=4096, dtype="bf16", bias=False, ignore=0.0,
             weighted=False),
        # all tensors of a small model, binary16, parameters and gradients in
        # one flat bucket each: tensors start at any element
        dict(name="adamw_small", op="adamw", layers=2, N=1000, K=264, param="f16", grad="f16", copy="none", bits=32,
             flat=True),
        # FP32 master weights of two blocks, bfloat16 gradients and the
        # bfloat16 copies that the next forward pass reads
        dict(name="adamw_masters", op="adamw", layers=2, N=14336, K=4096, param="f32", grad="bf16", copy="bf16",
             bits=32, flat=False),
        # odd sizes with states in 8 bits: blocks that end inside a tensor
        dict(name="adamw8_ragged", op="adamw", layers=1, N=1000, K=770, param="bf16", grad="f32", copy="none", bits=8,
             flat=True),
        # four blocks in bfloat16 with states in 8 bits
        dict(name="adamw8_blocks", op="adamw", layers=4, N=14336, K=4096, param="bf16", grad="bf16", copy="none",
             bits=8, flat=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Log-uniform; a third are multiples of 64, a third of 8, a third any."""
    v = _logint(rng, lo, hi)
    step = rng.choice((64, 8, 1))
    return max(lo, min(hi, v // step * step or step))


def draw(rng):
    op = rng.choice(("loss", "loss_bwd", "adamw"))
    if op == "adamw":
        param = rng.choice(("f16", "bf16", "f32"))
        return dict(op=op, layers=rng.randint(1, 4), N=_size(rng, 64, 14336), K=_size(rng, 64, 4096), param=param,
                    grad=rng.choice((param, "f32", "bf16")),
                    copy=rng.choice(("none", "bf16", "f16")) if param == "f32" else "none", bits=rng.choice((32, 8)),
                    flat=rng.random() < 0.5)
    # a third single tokens and small batches, the rest up to the training step's rows
    M = _logint(rng, 1, 16) if rng.random() < 0.34 else _size(rng, 17, 8192)
    case = dict(op=op, M=M, V=_size(rng, 512, 131072), K=_size(rng, 64, 4096), dtype=rng.choice(("f16", "bf16")),
                bias=rng.random() < 0.5, ignore=rng.choice((0.0, 0.1, 0.5)))
    case["save" if op == "loss" else "weighted"] = rng.random() < 0.5
    return case


def _shapes(case):
    """Three weights and a bias a layer."""
    N, K = case["N"], case["K"]
    return [(N, K), (N, K), (K, N), (N,)] * case["layers"]


def _tensors(shapes, dt, flat):
    """Empty tensors; with `flat`, views of one buffer, each at the element where the last one ended."""
    if not flat:
        return [torch.empty(s, dtype=dt, device=_DEV) for s in shapes]
    sizes = [math.prod(s) for s in shapes]
    return [t.view(s) for t, s in zip(torch.empty(sum(sizes), dtype=dt, device=_DEV).split(sizes), shapes)]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed))

    def normal(shape, std=1.0, dt=torch.float32):
        return (torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32) * std).to(dt)

    if case["op"] == "adamw":
        shapes, small = _shapes(case), case["bits"] == 8
        st = dict(case=case, p=_tensors(shapes, _DT[case["param"]], case["flat"]),
                  g=_tensors(shapes, _DT[case["grad"]], case["flat"]), m=[], v=[], ms=[], vs=[], copy=None)
        for p, g in zip(st["p"], st["g"]):
            p.copy_(normal(p.shape, 0.02))
            # gradients of a few hundred steps: their size differs from element to element
            size = 1e-3 * torch.exp(normal(p.shape))
            g.copy_(normal(p.shape) * size)
            m, v = normal(p.shape) * (0.25 * size), size.square() * (0.75 + 0.25 * normal(p.shape).square())
            if small:
                m, ms = _codes(m.flatten(), True)
                v, vs = _codes(v.flatten().sqrt(), False)
                st["ms"].append(ms)
                st["vs"].append(vs)
                m, v = m.view(p.shape), v.view(p.shape)
            st["m"].append(m)
            st["v"].append(v)
        if case["copy"] != "none":
            st["copy"] = [p.to(_DT[case["copy"]]) for p in st["p"]]
        return st
    M, V, K, dt = case["M"], case["V"], case["K"], _DT[case["dtype"]]
    st = dict(case=case, x=normal((M, K), 1.0, dt), w=normal((V, K), 0.02, dt),
              b=normal((V,), 0.1, dt) if case["bias"] else None)
    t = torch.randint(0, V, (M,), generator=gen, device=_DEV)
    st["t"] = torch.where(torch.rand(M, generator=gen, device=_DEV) < case["ignore"], _IGNORE, t)
    if case["op"] == "loss_bwd":
        st["lse"] = _lse(_logits(st))
        # a mean over the rows; binary16 gradients carry a loss scale
        mean = torch.full((1,), (1024.0 if case["dtype"] == "f16" else 1.0) / M, device=_DEV)
        st["dloss"] = mean * (0.5 + torch.rand(M, generator=gen, device=_DEV)) if case["weighted"] else mean.expand(M)
    return st


# ---- plain forms: elementary operations in 32 bits --------------------------
def _logits(st):
    z = st["x"].float() @ st["w"].float().T
    return z if st["b"] is None else z + st["b"].float()


def _lse(z):
    top = z.amax(1)
    return top + (z - top[:, None]).exp_().sum(1).log()


def _blocks(a):
    """A flat tensor as rows of a scale's elements, the last filled up with zeros."""
    return torch.nn.functional.pad(a, (0, -a.numel() % _BLOCK)).view(-1, _BLOCK)


def _codes(a, signed):
    """Codes and scales of a flat tensor: a = scale c |c|, c the nearest integer to +-sqrt(|a| / scale)."""
    top = 127.0 if signed else 255.0
    r = _blocks(a)
    most = r.abs().amax(1, keepdim=True)
    inv = torch.where(most > 0, most.reciprocal() * (top * top), 0.0)
    y = r.abs() * inv
    c = y.sqrt().floor()
    c = c + (y > c * c + c + 0.25)  # y > (c + 1/2)^2
    if signed:
        c = c * r.sign()
    else:
        c = torch.where(r > 0, c.clamp(min=1.0), c)  # what is not zero stays so
    code = c.to(torch.int8 if signed else torch.uint8).flatten()[:a.numel()]
    return code, (most * (1.0 / (top * top))).flatten()


def _value(code, scale):
    c = _blocks(code.flatten().float())
    return (scale[:, None] * (c * c.abs())).flatten()[:code.numel()].view(code.shape)


def _moments(st, i):
    if st["case"]["bits"] == 32:
        return st["m"][i], st["v"][i]
    return _value(st["m"][i], st["ms"][i]), _value(st["v"][i], st["vs"][i]).square()


def _plain_adamw(st, i):
    """Updates the i-th tensor and its state; returns them."""
    g, p = st["g"][i].float(), st["p"][i].float()
    m, v = _moments(st, i)
    m = m * _B1 + g * (1.0 - _B1)
    v = v * _B2 + (g * g) * (1.0 - _B2)
    root = v.sqrt()
    step = m / (root * (1.0 / math.sqrt(1.0 - _B2 ** _STEP)) + _EPS)
    p = p * (1.0 - _LR * _WD) - step * (_LR / (1.0 - _B1 ** _STEP))
    out = [st["p"][i].copy_(p)]
    if st["copy"] is not None:
        out.append(st["copy"][i].copy_(p))
    if st["case"]["bits"] == 32:
        return out + [st["m"][i].copy_(m), st["v"][i].copy_(v)]
    for name, a, signed in (("m", m, True), ("v", root, False)):
        code, scale = _codes(a.flatten(), signed)
        st[name][i].copy_(code.view(p.shape))
        st[name + "s"][i].copy_(scale)
    return out + list(_moments(st, i))


def _plain(st):
    case = st["case"]
    if case["op"] == "adamw":
        return [t for i in range(len(st["p"])) for t in _plain_adamw(st, i)]
    z = _logits(st)
    used = st["t"] != _IGNORE
    t = torch.where(used, st["t"], 0)
    rows = torch.arange(len(t), device=z.device)
    if case["op"] == "loss":
        lse = _lse(z)
        loss = torch.where(used, lse - z[rows, t], 0.0)
        return [loss, lse] if case["save"] else [loss]
    dt = _DT[case["dtype"]]
    q = z.sub_(st["lse"][:, None]).exp_()
    q[rows, t] -= 1.0
    q *= torch.where(used, st["dloss"], 0.0)[:, None]
    out = [(q @ st["w"].float()).to(dt), (q.T @ st["x"].float()).to(dt)]
    return out + ([q.sum(0).to(dt)] if case["bias"] else [])


# ---- the framework's entry points -------------------------------------------
def _own(st):
    import linear_fp16_gb300 as L
    case = st["case"]
    if case["op"] == "loss":
        out = L.linear_cross_entropy(st["x"], st["w"], st["t"], st["b"], ignore_index=_IGNORE, save=case["save"])
        return list(out) if case["save"] else [out]
    if case["op"] == "loss_bwd":
        out = L.linear_cross_entropy_backward(st["dloss"], st["x"], st["w"], st["t"], st["lse"], st["b"],
                                              ignore_index=_IGNORE, need_db=case["bias"])
        return [t for t in out if t is not None]
    state = L.AdamWState(st["m"], st["v"], st["ms"], st["vs"])
    L.adamw_step(st["p"], st["g"], state, step=_STEP, lr=_LR, betas=(_B1, _B2), eps=_EPS, weight_decay=_WD,
                 copies=st["copy"])
    m, v = state.values() if case["bits"] == 8 else (st["m"], st["v"])
    parts = [st["p"], m, v] if st["copy"] is None else [st["p"], st["copy"], m, v]
    return [t for group in zip(*parts) for t in group]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        p, g = _DT[case["param"]].itemsize, _DT[case["grad"]].itemsize
        copy = 0 if case["copy"] == "none" else 2
        # states read and written; those in 8 bits with their scales, and returned in 32
        state = 16 if case["bits"] == 32 else 4 + 16 / _BLOCK + 8
        return {"bytes": n * (2 * p + g + copy + state), "flops": 14 * n}
    M, V, K, b = case["M"], case["V"], case["K"], int(case["bias"])
    if case["op"] == "loss":
        return {"bytes": 2 * (M * K + V * K + b * V) + M * (16 if case["save"] else 12), "flops": 2 * M * V * K}
    return {"bytes": 2 * (2 * M * K + 2 * V * K + 2 * b * V) + M * (16 if case["weighted"] else 12),
            "flops": 6 * M * V * K}


# ---- the definitions in 64 bits ----------------------------------------------
def _exact_adamw(st, case):
    res = []
    for i, (p, g) in enumerate(zip(st["p"], st["g"])):
        g = g.double()
        if case["bits"] == 8:
            # scale of every element
            ms, vs = (s.double().repeat_interleave(_BLOCK)[:p.numel()].view(p.shape) for s in (st["ms"][i], st["vs"][i]))
            cm, cv = st["m"][i].double(), st["v"][i].double()
            m, v = ms * cm * cm.abs(), (vs * cv.pow(2)).pow(2)
        else:
            m, v = st["m"][i].double(), st["v"][i].double()
        m = _B1 * m + (1 - _B1) * g
        v = _B2 * v + (1 - _B2) * g.square()
        mhat, vhat = m / (1 - _B1 ** _STEP), v / (1 - _B2 ** _STEP)
        new = p.double() * (1 - _LR * _WD) - _LR * mhat / (vhat.sqrt() + _EPS)
        if case["bits"] == 8:
            # which code a value next to a border gets is its 32-bit rounding's
            # matter: one element in 10^5 gets another one from 64 bits
            m = v = None
        res += [new, m, v] if st["copy"] is None else [new, new, m, v]
    return res


def exact(case, seed):
    if case["op"] != "adamw" and work(case)["flops"] > 1.2e13:
        return None  # minutes in 64 bits
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(st, case)
    x, w, t, V = st["x"].double(), st["w"].double(), st["t"], case["V"]
    b = torch.zeros(V, dtype=torch.float64, device=_DEV) if st["b"] is None else st["b"].double()
    keep = (t >= 0).double()
    lab = t.clamp(min=0).unsqueeze(1)
    step = max(1, 2 ** 27 // V)  # rows at a time
    spans = [slice(i, i + step) for i in range(0, case["M"], step)]
    if case["op"] == "loss":
        loss, lse = [], []
        for r in spans:
            z = torch.addmm(b, x[r], w.t())
            lse.append(torch.logsumexp(z, dim=1))
            loss.append((lse[-1] - z.gather(1, lab[r]).squeeze(1)) * keep[r])
        return [torch.cat(loss), torch.cat(lse)] if case["save"] else [torch.cat(loss)]
    dx, dw, db = [], torch.zeros_like(w), torch.zeros_like(b)
    for r in spans:
        q = torch.exp(torch.addmm(b, x[r], w.t()) - st["lse"][r].double().unsqueeze(1))
        q.scatter_add_(1, lab[r], torch.full_like(lab[r], -1, dtype=torch.float64))
        q *= (keep[r] * st["dloss"][r].double()).unsqueeze(1)
        dx.append(q @ w)
        dw.addmm_(q.t(), x[r])
        db += q.sum(dim=0)
    return [torch.cat(dx), dw] + ([db] if case["bias"] else [])

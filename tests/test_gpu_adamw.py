"""The AdamW step: against its FP32 definition bit for bit, and against 64 bits.

The step's numerics are FP32 operations rounded one by one in a stated order, so
the same operations in torch on the CPU (one rounding each) give its bits, 8-bit codes
among them.  Against 64 bits, with u = 2^-24 and the first-order sums of the roundings on the way:
* m: the products round twice each (constant and product), the sum once;
* v: the same, with g^2 once more;
* the update m / (sqrt(v) c + eps): sqrt halves v's relative error and each of five
  operations adds u, the factors' own rounding two more.
"""
import math

import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}
SIZES = [1, 3, 4, 255, 256, 257, 1000, 4099, 65537, 300000]
HYPER = dict(step=7, lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
NAMES = ("m", "v", "m_scale", "v_scale")


def blocks(a):
    return torch.nn.functional.pad(a, (0, -a.numel() % 256)).view(-1, 256)


def encode(a, top):
    """Codes and scales of a flat FP32 tensor, as include/poot_train.h states them."""
    r = blocks(a)
    most = r.abs().amax(1, keepdim=True)
    bad, none = ~r.isfinite().all(1, keepdim=True), most < 2.0 ** -110
    inv = torch.where(bad | none, 0.0, most.reciprocal() * float(top * top))
    y = r.abs() * inv
    c = y.sqrt().floor()
    c = (c + (y > c * c + c + 0.25)).nan_to_num(0.0)
    c = torch.where(r < 0, -c, c) if top == 127 else torch.where(r > 0, c.clamp(min=1), c)
    scale = torch.where(none, 0.0, most * (1.0 / (top * top)))
    scale = torch.where(bad, math.nan, scale)
    return c.to(torch.int8 if top == 127 else torch.uint8).flatten()[:a.numel()], scale.flatten()


def decode(code, scale):
    c = blocks(code.flatten().float())
    return (scale[:, None] * (c * c.abs())).flatten()[:code.numel()].view(code.shape)


def moments(st):
    if len(st) == 2:
        return st
    m, v, ms, vs = st
    return decode(m, ms), decode(v, vs).square()


def reference(p, g, st, *, step, lr, betas, eps, weight_decay, grad_scale=1.0, dt64=False):
    """New (p before its rounding, m, v, sqrt(v), the update) in FP32, rounded one by one; in 64 bits with dt64."""
    f = (lambda t: t.double()) if dt64 else (lambda t: t.float())
    m, v = (f(t) for t in moments(st))
    g = f(g) * grad_scale
    m = m * betas[0] + g * (1.0 - betas[0])
    v = v * betas[1] + (g * g) * (1.0 - betas[1])
    root = v.sqrt()
    c = 1.0 / math.sqrt(-math.expm1(step * math.log(betas[1]))) if betas[1] else 1.0
    s = lr / -math.expm1(step * math.log(betas[0])) if betas[0] else lr
    q = m / (root * c + eps)
    return f(p) * (1.0 - lr * weight_decay) - q * s, m, v, root, q * s


def make(sizes, pd, gd, bits, seed, flat=False):
    """(params, grads, states) on the CPU, and the same on the GPU."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda s: torch.randn(s, generator=gen)
    p = [(n(s) * 0.1).to(pd) for s in sizes]
    g = [(n(s) * torch.exp(n(s)) * 1e-2).to(gd) for s in sizes]
    st = []
    for s in sizes:
        m, v = n(s) * 3e-3, (n(s) * 1e-2).square()
        if bits == 8:
            (cm, sm), (cv, sv) = encode(m, 127), encode(v.sqrt(), 255)
            st.append((cm, cv, sm, sv))
        else:
            st.append((m, v))

    def up(ts):
        if not flat:
            return [t.to(DEV) for t in ts]
        buf = torch.empty(1 + sum(t.numel() for t in ts), dtype=ts[0].dtype, device=DEV)
        return [b.copy_(t) for b, t in zip(buf[1:].split([t.numel() for t in ts]), ts)]
    state = L.AdamWState(*(up([s[i] for s in st]) for i in range(2 if bits == 32 else 4)))
    return (p, g, st), (up(p), up(g), state)


def lists(state):
    return [state.m, state.v] if state.bits == 32 else [state.m, state.v, state.m_scale, state.v_scale]


def state_of(state, i):
    return [t[i].cpu() for t in lists(state)]


def same(a, b):
    if not a.is_floating_point():
        return torch.equal(a, b)
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def check_bits(host, dev, copies=None, **hyper):
    (p, g, st), (dp, dg, state) = host, dev
    for i in range(len(p)):
        new, m, v, root, _ = reference(p[i], g[i], st[i], **hyper)
        assert same(dp[i].cpu(), new.to(p[i].dtype)), (i, "p")
        if state.bits == 32:
            want = (m, v)
        else:
            (cm, sm), (cv, sv) = encode(m, 127), encode(root, 255)
            want = (cm, cv, sm, sv)
        have = state_of(state, i)
        for k in range(0 if state.bits == 32 else 2):
            # (a block that reads as NaN does so whatever its codes)
            off = want[k + 2].isnan().repeat_interleave(256)[:want[k].numel()]
            have[k][off] = want[k][off] = 0
        for got, ref, name in zip(have, want, NAMES):
            assert same(got, ref), (i, name, int((got != ref).sum()), got.numel())
        if copies is not None and copies[i] is not None:
            assert same(copies[i].cpu(), new.to(copies[i].dtype)), (i, "copy")


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gd", list(DT))
@pytest.mark.parametrize("pd", list(DT))
def test_bits_of_the_definition(pd, gd, bits, flat):
    host, dev = make(SIZES, DT[pd], DT[gd], bits, 1, flat)
    L.adamw_step(*dev, **HYPER)
    check_bits(host, dev, **HYPER)


@pytest.mark.parametrize("pd", list(DT))
def test_against_64_bits(pd):
    dt = DT[pd]
    host, dev = make(SIZES, dt, dt, 32, 2)
    L.adamw_step(*dev, **HYPER)
    b1, b2 = HYPER["betas"]
    for i, (p, g, st) in enumerate(zip(*host)):
        new, m, v, _, update = reference(p, g, st, dt64=True, **HYPER)
        gm, gv = state_of(dev[2], i)
        em = U * (2 * (b1 * st[0]).abs() + 3 * ((1 - b1) * g.double()).abs() + m.abs()) * 1.01
        ev = U * (2 * b2 * st[1] + 4 * (1 - b2) * g.double().square() + v) * 1.01 + 2.0 ** -149
        assert bool(((gm - m).abs() <= em).all()) and bool(((gv - v).abs() <= ev).all())
        eu = update.abs() * (ev / (2 * v).clamp_min(1e-300) + 8 * U) + em / m.abs().clamp_min(1e-300) * update.abs()
        e = eu + 2 * U * p.double().abs() + U * new.abs()
        assert bool(((dev[0][i].cpu().double() - new).abs() <= e + (new.abs() + e) * EPS[dt] + TINY[dt]).all())


def test_codes_are_nearest_and_values_are_what_they_stand_for():
    host, dev = make(SIZES, torch.float32, torch.float32, 8, 3)
    L.adamw_step(*dev, **HYPER)
    vm, vv = dev[2].values()
    for i, (p, g, st) in enumerate(zip(*host)):
        _, m, v, root, _ = reference(p, g, st, dt64=True, **HYPER)
        cm, cv, sm, sv = state_of(dev[2], i)
        assert torch.equal(vm[i].cpu(), decode(cm, sm)) and torch.equal(vv[i].cpu(), decode(cv, sv).square())
        for a, c, s, top in ((m, cm, sm, 127), (root, cv, sv, 255)):
            most = blocks(a.flatten()).abs().amax(1)
            assert bool(((s.double() * top * top - most).abs() <= most * 2.0 ** -21).all())
            y = (blocks(a.flatten()).abs() / most[:, None]).sqrt() * top
            # half a code, and what FP32 leaves open: 2^-21 of sqrt(y)
            far = (y - blocks(c.float().flatten()).abs()).abs()
            assert bool((far[y > 0.5] <= 0.5 + 255 * 2.0 ** -21).all())
            assert float(blocks(c.float().flatten()).abs().amax(1).min()) == top
        assert bool((cv[root.flatten() > 0] >= 1).all())


def test_roots_and_quotients_are_rounded_to_nearest():
    """Every significand of v (1 <= v < 4: powers of 4 only shift the exponent) and
    many of m: with g = 0, betas of 1/2 and factors of 1 the step leaves p = -m / sqrt(v)."""
    v = torch.arange(0x3f800000, 0x40800000, device=DEV, dtype=torch.int64).to(torch.int32).view(torch.float32)
    gen = torch.Generator(device=DEV).manual_seed(12)
    for exponent in (0, -90, 90):
        for m in (torch.ones_like(v), torch.randn(v.shape, generator=gen, device=DEV),
                  torch.randn(v.shape, generator=gen, device=DEV) * 1e-3):
            p, s = torch.zeros_like(v), v * 2.0 ** exponent
            L.adamw_step([p], [torch.zeros_like(v)], L.AdamWState([2 * m], [2 * s]), step=2 ** 40, lr=1.0,
                         betas=(0.5, 0.5), eps=0.0, weight_decay=0.0)
            assert torch.equal(p, -(m / s.sqrt()))


def test_codes_of_every_reciprocal():
    """A block's largest value, of every significand, decides its codes through its
    reciprocal: 65536 significands a pass, each with 255 values spread below it."""
    gen = torch.Generator().manual_seed(14)
    below = torch.rand(255, generator=gen).square()
    for part in (0, 37, 77, 127):
        top = (torch.arange(1 << 16) + (part << 16) + 0x3f800000).to(torch.int32).view(torch.float32)
        m = torch.cat([top[:, None], top[:, None] * below], 1).flatten()
        v = m.square()
        m8 = L.AdamWState([torch.zeros(m.numel(), dtype=torch.int8, device=DEV)],
                          [torch.zeros(m.numel(), dtype=torch.uint8, device=DEV)],
                          [torch.zeros(1 << 16, device=DEV)], [torch.zeros(1 << 16, device=DEV)])
        # from a state of zeros with betas of 0 the averages are g and g^2
        p = [torch.zeros(m.numel(), device=DEV)]
        L.adamw_step(p, [m.to(DEV)], m8, step=1, lr=0.0, betas=(0.0, 0.0), eps=1.0, weight_decay=0.0)
        (cm, sm), (cv, sv) = encode(m, 127), encode(v.sqrt(), 255)
        for got, ref in zip(state_of(m8, 0), (cm, cv, sm, sv)):
            assert torch.equal(got, ref), part


@pytest.mark.parametrize("bits", [32, 8])
def test_copies_of_master_weights(bits):
    host, dev = make([300, 4096, 77, 1000], torch.float32, torch.bfloat16, bits, 4)
    copies = [torch.empty(300, dtype=torch.bfloat16, device=DEV), torch.empty(4096, dtype=torch.float16, device=DEV), None,
              torch.empty(1003, dtype=torch.bfloat16, device=DEV)[3:]]
    decays = [0.0, 0.1, 0.3, 0.0]
    L.adamw_step(*dev, **{**HYPER, "weight_decay": decays}, copies=copies)
    for i in range(4):
        check_bits(tuple([t[i]] for t in host), ([dev[0][i]], [dev[1][i]], L.AdamWState(*([t[i]] for t in lists(dev[2])))),
                   [copies[i]], **{**HYPER, "weight_decay": decays[i]})


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_and_extreme_numbers(bits):
    for hyper in (dict(step=1, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0),
                  dict(step=2 ** 40, lr=0.0, betas=(0.0, 0.0), eps=1.0, weight_decay=2.0),
                  dict(step=3, lr=1.0, betas=(0.5, 0.25), eps=0.0, weight_decay=0.5, grad_scale=2.0 ** -10)):
        p = [torch.randn(700)]
        g = torch.randn(700)
        g[:5] = torch.tensor([1e25, 1e-30, 1e-44, -0.0, 3e38])
        g[256:512] = 0.0
        g[600:] *= 1e-41
        zero = L.adamw_state([t.to(DEV) for t in p], bits=bits)
        host = (p, [g], [tuple(state_of(zero, 0))])
        dev = ([p[0].to(DEV)], [g.to(DEV)], zero)
        L.adamw_step(*dev, **hyper)
        check_bits(host, dev, **hyper)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_finite_stays_in_its_element_or_block(bad):
    for bits in (32, 8):
        host, dev = make([1000], torch.float32, torch.float32, bits, 5)
        dev[1][0][300] = bad
        L.adamw_step(*dev, **HYPER)
        m, v = dev[2].values()
        hit = torch.zeros(1000, dtype=torch.bool)
        hit[300 if bits == 32 else slice(256, 512)] = True
        for t in (m[0].cpu(), v[0].cpu()):
            assert bool(t[~hit].isfinite().all()) and not bool(t[hit].isfinite().any())
        p = dev[0][0].cpu()
        assert bool(p.isnan()[300]) and int(p.isnan().sum()) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_long_lists(bits):
    sizes = [(i * 37) % 700 for i in range(900)]    # several launches, empty ones among them
    host, dev = make(sizes, torch.bfloat16, torch.float32, bits, 6)
    L.adamw_step(*dev, **HYPER)
    check_bits(host, dev, **HYPER)
    if bits == 8:
        for got, c, s in zip(dev[2].values()[0], dev[2].m, dev[2].m_scale):
            assert torch.equal(got.cpu(), decode(c.cpu(), s.cpu()))


@pytest.mark.parametrize("bits", [32, 8])
def test_factors_on_the_device_and_graphs(bits):
    """lr, step and grad_scale as tensors: the host's bits, and a captured step
    that follows them from replay to replay."""
    hyper = {**HYPER, "weight_decay": 0.0}
    _, dev = make(SIZES, torch.float32, torch.bfloat16, bits, 7)
    _, want = make(SIZES, torch.float32, torch.bfloat16, bits, 7)
    _, graphed = make(SIZES, torch.float32, torch.bfloat16, bits, 7)
    step = torch.tensor(0, device=DEV)
    lr, scale = torch.tensor([0.0], device=DEV), torch.tensor(0.25, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step.add_(1)
        L.adamw_step(*graphed, **{**hyper, "step": step, "lr": lr, "grad_scale": scale})
    for t in range(1, 4):
        rate = float(torch.tensor(1e-3 * t))
        lr.fill_(rate)
        L.adamw_step(*want, **{**hyper, "step": t, "lr": rate, "grad_scale": 0.25})
        g.replay()
        L.adamw_step(*dev, **{**hyper, "step": torch.tensor([t], device=DEV), "lr": lr, "grad_scale": scale})
        for i in range(len(SIZES)):
            for other in (dev, graphed):
                assert torch.equal(other[0][i], want[0][i]), (t, i)
                assert all(torch.equal(a, b) for a, b in zip(state_of(other[2], i), state_of(want[2], i))), (t, i)
    # weight decay: 1 - lr wd of two FP32 numbers, rounded once
    _, a = make([1000], torch.float32, torch.bfloat16, bits, 8)
    p0 = a[0][0].clone()
    a[1][0].zero_()
    a[2].m[0].zero_()
    L.adamw_step(*a, step=1, lr=torch.tensor(0.1, device=DEV), weight_decay=0.3)
    factor = 1.0 - float(torch.tensor(0.1)) * float(torch.tensor(0.3))
    assert torch.equal(a[0][0], p0 * float(torch.tensor(factor, dtype=torch.float64).float()))


def test_streams_versions_and_autograd_leaves():
    host, dev = make([5000, 100], torch.float32, torch.float32, 8, 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = dev[0][0].requires_grad_()
    before = p._version, dev[2].m[0]._version, dev[1][0]._version
    L.adamw_step(*dev, **HYPER, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert (p._version, dev[2].m[0]._version, dev[1][0]._version) == (before[0] + 1, before[1] + 1, before[2])
    p.requires_grad_(False)
    check_bits(host, dev, **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_is_written_outside(bits):
    n, band = 1003, 64
    host, dev = make([n], torch.bfloat16, torch.bfloat16, bits, 10)
    guarded = []

    def inside(t):
        b = torch.full((t.numel() + 2 * band,), 77, dtype=t.dtype, device=DEV)
        guarded.append(b)
        return b[band:-band].copy_(t)
    dev = ([inside(dev[0][0])], dev[1], L.AdamWState(*([inside(t[0])] for t in lists(dev[2]))))
    L.adamw_step(*dev, **HYPER)
    check_bits(host, dev, **HYPER)
    assert all(bool((b[:band] == 77).all()) and bool((b[-band:] == 77).all()) for b in guarded)


def test_refusals():
    _, (p, g, s) = make([512, 30], torch.float32, torch.bfloat16, 32, 11)
    _, (_, _, s8) = make([512, 30], torch.float32, torch.bfloat16, 8, 11)
    ok = dict(step=1)
    for args in (([p[0].double(), p[1]], g, s), (p, [g[0].int(), g[1]], s), (p, g, L.AdamWState(s8.m, s8.v)),
                 (p, g, L.AdamWState(s.m, s.v, s8.m_scale, s8.v_scale)), (p, [g[0], None], s)):
        with pytest.raises(TypeError):
            L.adamw_step(*args, **ok)
    for args in ((p, g[::-1], s), (p, g[:1], s), ([p[0].view(2, 256).t(), p[1]], g, s), ([p[0].cpu(), p[1]], g, s),
                 (p, g, L.AdamWState(s.m[:1], s.v)), (p, g, L.AdamWState(s8.m, s8.v, s8.v_scale[::-1], s8.v_scale))):
        with pytest.raises(ValueError):
            L.adamw_step(*args, **ok)
    for kw in (dict(copies=[p[0], None]), dict(step=torch.ones(1, device=DEV)), dict(lr=torch.ones(1, device=DEV).double())):
        with pytest.raises(TypeError):
            L.adamw_step(p, g, s, **{**ok, **kw})
    for kw in (dict(copies=[None]), dict(weight_decay=[0.1]), dict(lr=torch.ones(2, device=DEV)), dict(lr=torch.ones(1))):
        with pytest.raises(ValueError):
            L.adamw_step(p, g, s, **{**ok, **kw})
    before = [t.clone() for t in (*p, *s.m)]
    for kw in (dict(step=0), dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(eps=math.nan), dict(grad_scale=math.inf)):
        with pytest.raises(L.PootLinearError):
            L.adamw_step(p, g, s, **{**ok, **kw})
    with pytest.raises(L.PootLinearError):
        L.adamw_step([p[0], p[0]], [g[0], g[0]], L.AdamWState([s.m[0]] * 2, [s.v[0]] * 2), **ok)   # twice the same
    assert all(torch.equal(a, b) for a, b in zip(before, (*p, *s.m)))


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_beyond_2_to_the_31_elements(bits):
    n, tail = 2 ** 31 + 777, 5000
    p = [torch.zeros(n, dtype=torch.bfloat16, device=DEV)]
    g = [torch.zeros(n, dtype=torch.bfloat16, device=DEV)]
    state = L.adamw_state(p, bits=bits)
    cut = (n - tail) // 256 * 256
    gen = torch.Generator(device=DEV).manual_seed(13)
    p[0][cut:] = torch.randn(n - cut, generator=gen, device=DEV)
    g[0][cut:] = torch.randn(n - cut, generator=gen, device=DEV)
    small_p, small_g = [p[0][cut:].clone()], [g[0][cut:].clone()]
    small = L.adamw_state(small_p, bits=bits)
    L.adamw_step(p, g, state, **HYPER)
    L.adamw_step(small_p, small_g, small, **HYPER)
    assert torch.equal(p[0][cut:], small_p[0]) and not bool(p[0][:cut].any())
    for a, b in zip(lists(state), lists(small)):
        assert torch.equal(a[0][-b[0].numel():], b[0])

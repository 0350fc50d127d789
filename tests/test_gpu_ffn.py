"""The feed-forward operators on a GPU against plain 64-bit forms.

Bounds as derived in tests/ffn_ref.py.  Small-integer inputs make the
linear's gradients exact: bit-equality there.  Besides the elementwise bound,
results stay within u_p relative root-mean-square error (one rounding of the
result and one of dg, du, each about 0.42 u_p rms of a value).
"""
import pytest
import torch

import linear_fp16_gb300 as L
from tests import ffn_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F16, BF16 = torch.float16, torch.bfloat16
ACTS = ("silu", "gelu_tanh", "gelu_erf")


def _n(gen, shape, std, dt):
    return (torch.randn(shape, generator=gen) * std).to(dt)


def _gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * k for i, k in enumerate(key)))


def _ok():
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK


# sizes: one token to several tiles; odd everywhere; one wave to several; the
# pair and single-CTA tiles, their tails; K below, at and above one block
GATED = [
    (1, 64, 64), (1, 1, 1), (1, 5000, 512), (2, 264, 4096), (3, 77, 130), (8, 1000, 776), (16, 4096, 1024),
    (16, 33, 5), (17, 64, 64), (33, 200, 328), (64, 4096, 4096), (100, 130, 70), (128, 128, 64), (129, 65, 127),
    (200, 1000, 770), (256, 512, 2048), (257, 136, 1000), (300, 2056, 264), (700, 384, 96), (1024, 1024, 768),
    (2047, 1000, 770),
]


def _gated_inputs(M, N, K, dt, bias, seed=1):
    g = _gen(M, N, K, seed)
    std = 1.3 / max(1.0, K ** 0.5)
    return (_n(g, (M, K), 1.0, dt), _n(g, (N, K), std, dt), _n(g, (N, K), std, dt),
            _n(g, (N,), 0.1, dt) if bias else None, _n(g, (N,), 0.1, dt) if bias else None)


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _check_gated(x, wg, wu, bg, bu, act, save, got):
    dt = x.dtype
    refs, errs = R.gated64(x, wg, wu, bg, bu, act)
    outs = got if save else (got,)
    for o, r, e, name in zip(outs, refs, errs, "hgu"):
        R.check(o, r, e, name)
        if o.numel() >= 1000:
            R.rms(o, r, name, 2.0 ** -R.P[dt])


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("dt,act,bias,save", [(F16, "silu", True, False), (BF16, "gelu_erf", False, True),
                                              (F16, "gelu_tanh", True, True), (BF16, "silu", False, False)])
def test_gated_linear(M, N, K, dt, act, bias, save):
    ins = _gated_inputs(M, N, K, dt, bias)
    got = L.gated_linear(*_dev(*ins), activation=act, save=save)
    _ok()
    _check_gated(*ins, act, save, got)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 5, 11, 130, 520])
def test_gated_linear_extreme_gates(act, M):
    """Pre-activations from the far negative to the far positive tail."""
    N, K = 96, 16
    x = torch.zeros(M, K)
    x[:, 0] = torch.linspace(-300, 300, M) if M > 1 else -40.0
    x[:, 1] = 1.0
    wg = torch.zeros(N, K)
    wg[:, 0] = torch.linspace(0.01, 1.0, N)
    wu = torch.zeros(N, K)
    wu[:, 1] = torch.linspace(-2, 2, N)
    ins = [t.to(BF16) for t in (x, wg, wu)] + [None, None]
    got = L.gated_linear(*_dev(*ins), activation=act, save=True)
    _ok()
    assert all(torch.isfinite(t).all() for t in got)
    _check_gated(*ins, act, True, got)


@pytest.mark.parametrize("M", [1, 4, 16, 60, 300])
def test_gated_linear_row_pitch_and_offset_bases(M):
    """x as a column slice (any offset), weights halves of one tensor, out given."""
    N, K = 200, 136
    g = _gen(M, N, K, 5)
    wide = _n(g, (M, K + 24), 1.0, F16)
    w = _n(g, (2 * N, K), 0.1, F16)
    wd, dev_wide = w.to(DEV), wide.to(DEV)
    for off in (0, 8, 3):
        x = wide[:, off:off + K]
        out = torch.full((M, N), float("nan"), dtype=F16, device=DEV)
        got = L.gated_linear(dev_wide[:, off:off + K], wd[:N], wd[N:], out=out)
        _ok()
        assert got is out
        _check_gated(x, w[:N], w[N:], None, None, "silu", False, got)
    # weights that start at an odd element
    flat = _n(g, (2 * N * K + 1,), 0.1, F16)
    fd = flat.to(DEV)
    x = wide[:, :K].contiguous()
    wg, wu = flat[1:1 + N * K].view(N, K), flat[1 + N * K:].view(N, K)
    got = L.gated_linear(x.to(DEV), fd[1:1 + N * K].view(N, K), fd[1 + N * K:].view(N, K))
    _ok()
    _check_gated(x, wg, wu, None, None, "silu", False, got)


def test_gated_linear_one_bias_only():
    for M in (3, 200):
        ins = list(_gated_inputs(M, 72, 64, F16, True))
        for drop in (3, 4):
            use = list(ins)
            use[drop] = None
            got = L.gated_linear(*_dev(*use), save=True)
            _ok()
            _check_gated(*use, "silu", True, got)


def test_gated_linear_empty_sizes():
    z = lambda *s: torch.zeros(s, dtype=F16, device=DEV)
    assert L.gated_linear(z(0, 8), z(16, 8), z(16, 8)).shape == (0, 16)
    assert L.gated_linear(z(4, 8), z(0, 8), z(0, 8)).shape == (4, 0)
    bg = torch.linspace(-3, 3, 16).to(F16)
    bu = torch.linspace(2, -1, 16).to(F16)
    h, g, u = L.gated_linear(z(5, 0), z(16, 0), z(16, 0), bg.to(DEV), bu.to(DEV), save=True)
    _ok()
    assert torch.equal(g.cpu(), bg.expand(5, 16)) and torch.equal(u.cpu(), bu.expand(5, 16))
    ref = R.act64("silu", bg.double()) * bu.double()
    R.check(h, ref.expand(5, 16), R.ACT_ERR * ref.abs().expand(5, 16), "h")


def test_nan_and_inf_rows_stay_in_their_rows():
    for M in (4, 200):
        ins = list(_gated_inputs(M, 136, 128, F16, False))
        clean = L.gated_linear(*_dev(*ins))
        x = ins[0].clone()
        x[1, 3] = float("nan")
        x[2, 5] = float("inf")
        got = L.gated_linear(x.to(DEV), *_dev(*ins[1:]))
        _ok()
        assert torch.isnan(got[1]).all()
        assert not torch.isfinite(got[2]).any()
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])


# ---- gradients ------------------------------------------------------------------
BWD = [
    (1, 64, 64), (1, 1, 1), (3, 77, 130), (8, 1000, 776), (16, 512, 1024), (17, 64, 64), (65, 200, 328),
    (100, 130, 70), (128, 128, 64), (129, 65, 127), (333, 1000, 770), (256, 512, 2048), (257, 136, 1000),
    (700, 384, 96), (1024, 1024, 768), (64, 2048, 2048), (2048, 264, 512),
]


def _bwd_inputs(M, N, K, dt, seed=2):
    g = _gen(M, N, K, seed)
    std = 1.3 / max(1.0, K ** 0.5)
    return (_n(g, (M, N), 0.5, dt), _n(g, (M, K), 1.0, dt), _n(g, (N, K), std, dt), _n(g, (N, K), std, dt),
            _n(g, (M, N), 1.3, dt), _n(g, (M, N), 1.3, dt))


def _check_gated_bwd(ins, act, got):
    dh, x, wg, wu, g, u = ins
    dt = x.dtype
    (dg, du), (eg, eu) = R.gate_grad64(dh, g, u, act)
    xd, wgd, wud = x.double(), wg.double(), wu.double()
    dx, dwg, dwu, dbg, dbu = got
    checks = []
    if dx is not None:
        checks.append((dx, dg @ wgd + du @ wud,
                       R.product_bound(dg, eg, wgd, dt) + R.product_bound(du, eu, wud, dt)
                       + R.acc_err(2 * wg.shape[0]) * (dg.abs() @ wgd.abs() + du.abs() @ wud.abs()), "dx"))
    for o, d, e, name in ((dwg, dg, eg, "dwg"), (dwu, du, eu, "dwu")):
        if o is not None:
            checks.append((o, d.T @ xd, R.product_bound(d.T.contiguous(), e.T.contiguous(), xd, dt), name))
    for o, d, e, name in ((dbg, dg, eg, "dbg"), (dbu, du, eu, "dbu")):
        if o is not None:
            # at most M / 8 + 16 FP32 additions on the way of any term
            checks.append((o, d.sum(0), e.sum(0) + (d.shape[0] + 16) * 2.0 ** -24 * d.abs().sum(0), name))
    for o, r, e, name in checks:
        R.check(o, r, e, name)
        if o.numel() >= 1000:
            R.rms(o, r, name, 2.0 ** -R.P[dt])


@pytest.mark.parametrize("M,N,K", BWD)
@pytest.mark.parametrize("dt,act", [(F16, "silu"), (BF16, "gelu_tanh"), (F16, "gelu_erf")])
def test_gated_linear_backward(M, N, K, dt, act):
    ins = _bwd_inputs(M, N, K, dt)
    got = L.gated_linear_backward(*_dev(*ins), activation=act, need_db=True)
    _ok()
    _check_gated_bwd(ins, act, got)


@pytest.mark.parametrize("needs", [(True, False, False), (False, True, False), (False, False, True),
                                   (True, True, False), (False, False, False)])
def test_gated_linear_backward_subsets(needs):
    ins = _bwd_inputs(150, 136, 72, BF16)
    dev = _dev(*ins)
    full = L.gated_linear_backward(*dev, need_db=True)
    got = L.gated_linear_backward(*dev, need_dx=needs[0], need_dw=needs[1], need_db=needs[2])
    _ok()
    want = (needs[0], needs[1], needs[1], needs[2], needs[2])
    for o, f, w in zip(got, full, want):
        assert (o is not None) == w
        assert o is None or torch.equal(o, f)


@pytest.mark.parametrize("act", ACTS)
def test_gated_linear_backward_extreme_gates(act):
    M, N, K = 64, 72, 32
    ins = list(_bwd_inputs(M, N, K, BF16))
    ins[4] = torch.linspace(-300, 300, M * N).view(M, N).to(BF16)
    ins[4][0, :8] = torch.tensor([1e30, -1e30, 2e29, -2e29, 0.0, -0.0, 1e-38, -87.5]).to(BF16)
    got = L.gated_linear_backward(*_dev(*ins), activation=act, need_db=True)
    _ok()
    # cubes overflow FP32 there; value and slope are those of the limits
    assert not any(torch.isnan(t).any() for t in got)
    ins[4] = torch.linspace(-300, 300, M * N).view(M, N).to(BF16)
    got = L.gated_linear_backward(*_dev(*ins), activation=act, need_db=True)
    _ok()
    _check_gated_bwd(ins, act, got)


def test_gated_linear_backward_row_pitch():
    M, N, K = 90, 120, 88
    ins = _bwd_inputs(M, N, K, F16)
    views = []
    for i, t in enumerate(ins):
        if i in (2, 3):
            views.append(t.to(DEV))
            continue
        wide = torch.full((M, t.shape[1] + 13 + i), float("nan"), dtype=F16, device=DEV)
        wide[:, i + 1:i + 1 + t.shape[1]] = t.to(DEV)
        views.append(wide[:, i + 1:i + 1 + t.shape[1]])
    got = L.gated_linear_backward(*views, need_db=True)
    _ok()
    _check_gated_bwd(ins, "silu", got)


@pytest.mark.parametrize("M,N,K", BWD)
@pytest.mark.parametrize("dt", [F16, BF16])
def test_linear_backward_exact_on_small_integers(M, N, K, dt):
    """Sums of integer products below 2^24 are exact in FP32: one rounding."""
    g = _gen(M, N, K, 3)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(dt)
    dy, x, w = ints(M, N), ints(M, K), ints(N, K)
    dx, dw, db = L.linear_backward(*_dev(dy, x, w))
    _ok()
    for o, r in ((dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double()), (db, dy.double().sum(0))):
        assert torch.equal(o.cpu(), r.float().to(dt))


@pytest.mark.parametrize("M,N,K,dt", [(700, 384, 1000, F16), (2048, 520, 776, BF16), (9, 4096, 512, BF16)])
def test_linear_backward_normal_inputs(M, N, K, dt):
    g = _gen(M, N, K, 4)
    dy, x, w = _n(g, (M, N), 0.2, dt), _n(g, (M, K), 1.0, dt), _n(g, (N, K), 0.05, dt)
    dx, dw, db = L.linear_backward(*_dev(dy, x, w))
    _ok()
    z = torch.zeros(M, N, dtype=torch.float64)
    d = dy.double()
    R.check(dx, d @ w.double(), R.product_bound(d, z, w.double(), None), "dx")
    R.check(dw, d.T @ x.double(), R.product_bound(d.T, z.T, x.double(), None), "dw")
    R.check(db, d.sum(0), (M + 16) * 2.0 ** -24 * d.abs().sum(0), "db")


def test_backward_of_empty_sizes():
    t = lambda *s: torch.ones(s, dtype=F16, device=DEV)
    dx, dw, db = L.linear_backward(t(0, 16), t(0, 8), t(16, 8))
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    dx, dw, db = L.linear_backward(t(4, 0), t(4, 8), t(0, 8))
    assert not dx.any() and dw.shape == (0, 8)
    dx, dw, db = L.linear_backward(t(4, 16), t(4, 0), t(16, 0))
    assert dx.shape == (4, 0) and dw.shape == (16, 0) and bool((db == 4).all())
    out = L.gated_linear_backward(t(0, 16), t(0, 8), t(16, 8), t(16, 8), t(0, 16), t(0, 16), need_db=True)
    assert out[0].shape == (0, 8) and not any(o.any() for o in out[1:])
    out = L.gated_linear_backward(t(4, 0), t(4, 8), t(0, 8), t(0, 8), t(4, 0), t(4, 0), need_db=True)
    assert not out[0].any()
    _ok()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_match_differences(act):
    """dL/dv for L = sum dh * h against central differences of the 64-bit block.

    Step 1e-4 in 64 bits: the difference quotient is good to about 1e-7 of the
    gradient's scale, far below the results' own rounding.  dg, du and the
    results are rounded (2 u_p of the terms' magnitude sum bounds both)."""
    M, N, K = 24, 40, 32
    gen = _gen(M, N, K, 9)
    x, wg, wu, dh = (_n(gen, (M, K), 1.0, F16), _n(gen, (N, K), 0.2, F16), _n(gen, (N, K), 0.2, F16),
                     _n(gen, (M, N), 0.5, F16))
    bg, bu = _n(gen, (N,), 0.2, F16), _n(gen, (N,), 0.2, F16)
    dev = _dev(x, wg, wu, bg, bu)
    h, g, u = L.gated_linear(*dev, activation=act, save=True)
    got = L.gated_linear_backward(dh.to(DEV), *dev[:3], g, u, activation=act, need_db=True)
    _ok()
    p = [t.double() for t in (x, wg, wu, bg, bu)]
    loss = lambda q: float((dh.double() * R.act64(act, q[0] @ q[1].T + q[3]) * (q[0] @ q[2].T + q[4])).sum())
    # saved g and u carry one rounding each: their effect on dg, du is bounded
    # by u_p (|dg| + |du| + |dh|) times the largest curvature (< 2) and slope
    for i, (o, v) in enumerate(zip(got, p)):
        flat = o.detach().cpu().double().flatten()
        scale = float(flat.abs().max())
        for j in range(0, flat.numel(), max(1, flat.numel() // 7)):
            hi, lo = [t.clone() for t in p], [t.clone() for t in p]
            hi[i].view(-1)[j] += 1e-4
            lo[i].view(-1)[j] -= 1e-4
            fd = (loss(hi) - loss(lo)) / 2e-4
            assert abs(fd - float(flat[j])) <= 8 * 2.0 ** -11 * scale + 1e-6, (i, j)


def test_equal_calls_give_equal_bits():
    ins = _dev(*_bwd_inputs(600, 520, 264, BF16))
    a = L.gated_linear_backward(*ins, need_db=True)
    b = L.gated_linear_backward(*ins, need_db=True)
    _ok()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_another_stream_and_in_a_graph():
    fwd = _gated_inputs(300, 264, 192, F16, True)
    dev = _dev(*fwd)
    bwd = _dev(*_bwd_inputs(300, 264, 190, F16))
    want_f = L.gated_linear(*dev, save=True)
    want_b = L.gated_linear_backward(*bwd, need_db=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = L.gated_linear(*dev, save=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want_f))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gf = L.gated_linear(*dev, save=True)
            gb = L.gated_linear_backward(*bwd, need_db=True)
            norm = L.clip_grad_norm(list(gb[1:]), 0.5)
    for _ in range(2):
        graph.replay()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(gf, want_f))
    assert torch.equal(gb[0], want_b[0])
    ref = torch.sqrt(sum(t.double().square().sum() for t in want_b[1:]))
    assert abs(float(norm) - float(ref)) <= 1e-6 * float(ref)


def test_outputs_and_inputs_beyond_31_bits_of_elements():
    """M * N above 2^31: rows at both ends and in the middle against the
    64-bit form (N odd: rows of every alignment, no TMA stores)."""
    M, N, K = 66000, 32769, 16
    gen = torch.Generator(device=DEV).manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=torch.float32)
    x, wg, wu = rnd(M, K).to(BF16), (rnd(N, K) * 0.3).to(BF16), (rnd(N, K) * 0.3).to(BF16)
    h, g, u = L.gated_linear(x, wg, wu, save=True)
    rows = [0, 1, M // 2, 65534, 65535, M - 2, M - 1]
    pick = lambda t: t[rows].cpu()
    _check_gated(pick(x), wg.cpu(), wu.cpu(), None, None, "silu", True, (pick(h), pick(g), pick(u)))
    dx = L.gated_linear_backward(h, x, wg, wu, g, u, need_dw=False)[0]
    _ok()
    ins = (pick(h), pick(x), wg.cpu(), wu.cpu(), pick(g), pick(u))
    _check_gated_bwd(ins, "silu", (pick(dx), None, None, None, None))


def test_gradients_over_many_rows():
    """dW and db over more rows than one row block or K range holds."""
    M, N, K = 70000, 24, 40
    gen = _gen(M, N, K, 6)
    ints = lambda *s: torch.randint(-2, 3, s, generator=gen).to(F16)
    dy, x, w = ints(M, N), ints(M, K), ints(N, K)
    dx, dw, db = L.linear_backward(*_dev(dy, x, w))
    _ok()
    for o, r in ((dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double()), (db, dy.double().sum(0))):
        assert torch.equal(o.cpu(), r.float().to(F16))


@pytest.mark.parametrize("M,N,ld", [(1, 3, 8), (5, 11, 16), (300, 230, 230), (300, 230, 232), (1000, 1001, 1008), (70, 8, 8)])
def test_bias_gradients_of_ragged_columns(M, N, ld):
    """Column counts that end inside a group of eight, alone and beside the
    products, at several pitches; what lies between rows is never used."""
    gen = _gen(M, N, ld, 7)
    ints = lambda *s: torch.randint(-3, 4, s, generator=gen).to(BF16)
    wide = torch.full((M, ld), float("nan"), dtype=BF16, device=DEV)
    dy, x, w = ints(M, N), ints(M, 24), ints(N, 24)
    wide[:, :N] = dy.to(DEV)
    want = dy.double().sum(0).float().to(BF16)
    db = L.linear_backward(wide[:, :N], *_dev(x, w), need_dx=False, need_dw=False)[2]
    both = L.linear_backward(wide[:, :N], *_dev(x, w))
    _ok()
    assert torch.equal(db.cpu(), want) and torch.equal(both[2].cpu(), want)
    assert torch.equal(both[0].cpu(), (dy.double() @ w.double()).float().to(BF16))


@pytest.mark.parametrize("N", [202, 204, 201, 200, 34, 36])
@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_output_rows_at_any_alignment(N, off):
    """Rows and bases of 2, 4, 8 and 16 bytes' alignment; nothing outside the
    output is written."""
    M, K, pad = 150, 72, 64
    x, wg, wu, bg, bu = _gated_inputs(M, N, K, BF16, True, seed=8)
    flat = torch.full((M * N + 2 * pad,), -7.0, dtype=BF16, device=DEV)
    out = flat[pad + off:pad + off + M * N].view(M, N)
    h = L.gated_linear(*_dev(x, wg, wu, bg, bu), out=out)
    saved = L.gated_linear(*_dev(x, wg, wu, bg, bu), save=True)
    _ok()
    _check_gated(x, wg, wu, bg, bu, "silu", True, saved)
    assert h is out and torch.equal(h, saved[0])
    assert (flat[:pad + off] == -7).all() and (flat[pad + off + M * N:] == -7).all()

"""The vocabulary head's loss and gradients against their 64-bit forms (head_ref)."""
import math
import threading

import pytest
import torch

import linear_fp16_gb300 as L

from .head_ref import IGNORE, check, grads64, loss64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float16, torch.bfloat16]
SIZES = [  # one of each, odd ones, tiles' edges, one and several chunks of K
    (1, 1, 1), (1, 1000, 64), (3, 7, 5), (16, 4096, 128), (17, 1003, 770), (130, 513, 1030), (128, 256, 1024),
    (300, 2049, 200), (1024, 1024, 768), (129, 40001, 72), (5, 300, 2500), (257, 255, 33), (2, 131, 9000),
    (600, 5000, 1000), (70, 64, 33000),
    (1, 50001, 200), (7, 70000, 64), (100, 9000, 520), (128, 20000, 264),   # few rows on a stream of W
]


def make(M, V, K, dt, bias=True, ignore=0.2, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + M * 7 + V * 3 + K)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)
    x = (n(M, K) * scale).to(dt)
    w = (n(V, K) * (1.5 / max(K, 1) ** 0.5)).to(dt)
    b = (n(V) * 0.3).to(dt) if bias else None
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    t = torch.where(torch.rand(M, generator=g, device=DEV) < ignore, IGNORE, t)
    dloss = torch.rand(M, generator=g, device=DEV) + 0.25
    return x, w, t, b, dloss


def check_loss(x, w, t, b):
    loss, lse = L.linear_cross_entropy(x, w, t, b, save=True)
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == lse.shape == t.shape
    ref, e, rlse, el = loss64(x, w, t, b)
    check(lse, rlse, el, "lse")
    check(loss, ref, e, "loss")
    assert bool((loss[t == IGNORE] == 0).all())
    return loss, lse


def check_grads(dloss, x, w, t, lse, b, **kw):
    need = {k: kw.get(k, True) for k in ("need_dx", "need_dw", "need_db")}
    got = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, **need)
    for out, (ref, e), name in zip(got, grads64(dloss, x, w, t, lse, b), ("dx", "dw", "db")):
        assert (out is not None) == need["need_" + name]
        if out is not None:
            assert out.dtype == x.dtype
            check(out, ref, e, name)
    return got


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,V,K", SIZES)
def test_loss(M, V, K, dt):
    for bias in (False, True):
        x, w, t, b, _ = make(M, V, K, dt, bias)
        loss, _ = check_loss(x, w, t, b)
        assert torch.equal(L.linear_cross_entropy(x, w, t, b), loss)  # with and without lse, and again


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,V,K", SIZES)
def test_gradients(M, V, K, dt):
    for bias in (False, True):
        x, w, t, b, dloss = make(M, V, K, dt, bias, seed=1)
        lse = loss64(x, w, t, b)[2].float()
        got = check_grads(dloss, x, w, t, lse, b)
        again = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        assert bool((got[0][t == IGNORE] == 0).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("M,V,K", [(2048, 70001, 64), (8300, 50000, 72), (4100, 100000, 8)])
def test_gradients_over_several_pieces_of_the_vocabulary(M, V, K, dt):
    x, w, t, b, dloss = make(M, V, K, dt, seed=2)
    lse = loss64(x, w, t, b)[2].float()
    got = check_grads(dloss, x, w, t, lse, b)
    again = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("need", ["need_dx", "need_dw", "need_db"])
@pytest.mark.parametrize("M,V,K", [(300, 1003, 130), (2048, 70001, 64)])
def test_each_gradient_alone_is_what_all_give(M, V, K, need):
    x, w, t, b, dloss = make(M, V, K, torch.bfloat16, seed=3)
    lse = loss64(x, w, t, b)[2].float()
    only = {k: k == need for k in ("need_dx", "need_dw", "need_db")}
    check_grads(dloss, x, w, t, lse, b, **only)


@pytest.mark.parametrize("dt", DTYPES)
def test_dloss_of_any_stride_and_size(dt):
    M, V, K = 200, 1000, 96
    x, w, t, b, dloss = make(M, V, K, dt, seed=4)
    lse = loss64(x, w, t, b)[2].float()
    wide = torch.rand(M, 3, device=DEV)
    for d in (torch.full((1,), 1 / M, device=DEV).expand(M), wide[:, 1], dloss * 2.0 ** -40 if dt == torch.bfloat16 else
              dloss * 2.0 ** -6, dloss * 1000, torch.zeros(M, device=DEV), -dloss,
              torch.where(torch.arange(M, device=DEV) % 3 == 0, 0.0, dloss)):
        check_grads(d, x, w, t, lse, b)


def test_small_probabilities_survive_in_binary16():
    """A flat softmax over 30000 columns: p is 3.3e-5, below binary16's normal
    range; with a mean over rows it would be below the smallest subnormal."""
    M, V, K = 64, 30000, 64
    x, w, t, _, _ = make(M, V, K, torch.float16, bias=False, ignore=0, seed=5)
    lse = loss64(x, w * 0, t, None)[2].float()
    dloss = torch.full((1,), 2.0 ** -10, device=DEV).expand(M)
    _, dw, db = L.linear_cross_entropy_backward(dloss * 2 ** 10, x, w * 0, t, lse, need_db=True)
    rest = torch.ones(V, dtype=torch.bool, device=DEV)
    rest[t] = False
    # db of a column without targets: M / V times dloss, each q rounded (2^-11) and the sum rounded
    assert float((db[rest].double() / (M / V) - 1).abs().max()) <= 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -19
    check_grads(dloss, x, w * 0, t, lse, None)


def test_gradients_against_differences():
    """The loss itself, moved along a direction of each input."""
    M, V, K = 96, 500, 64
    x, w, t, b, dloss = make(M, V, K, torch.bfloat16, seed=6)
    _, lse = L.linear_cross_entropy(x, w, t, b, save=True)
    got = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
    total = lambda *a: float((loss64(a[0], a[1], t, a[2])[0] * dloss).sum())
    args = [v.double() for v in (x, w, b)]
    g = torch.Generator(device=DEV).manual_seed(7)
    for i, d in enumerate(got):
        u = torch.randn(args[i].shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        plus, minus = [[v + s * h * u if j == i else v for j, v in enumerate(args)] for s in (1, -1)]
        slope = (total(*plus) - total(*minus)) / (2 * h)
        # two roundings to bfloat16 an element, at most 2^-8 of it each, along a random direction
        lim = 4 * 2.0 ** -8 * float(d.double().norm()) + 1e-6
        assert abs(slope - float((d.double() * u).sum())) <= lim, i


@pytest.mark.parametrize("M", [1, 40, 300])
def test_infinite_logits_follow_the_formula(M):
    V, K = 700, 64
    x, w, t, b, dloss = make(M, V, K, torch.bfloat16, ignore=0, seed=8)
    masked = b.clone()
    masked[::3] = -math.inf
    t = t // 3 * 3 + 1
    t = torch.where(t < V, t, 1)
    _, lse = check_loss(x, w, t, masked)
    dx, dw, db = check_grads(dloss, x, w, t, lse, masked)
    assert bool((dw[::3] == 0).all()) and bool((db[::3] == 0).all())
    assert bool(torch.isposinf(L.linear_cross_entropy(x, w, t * 0, masked)).all())      # a masked target
    loss, lse = L.linear_cross_entropy(x, w, t, torch.full_like(b, -math.inf), save=True)
    assert bool(torch.isneginf(lse).all()) and bool(loss.isnan().all())               # nothing left
    high = b.clone()
    high[5] = math.inf
    loss, lse = L.linear_cross_entropy(x, w, torch.full_like(t, 6), high, save=True)
    assert bool(torch.isposinf(lse).all()) and bool(torch.isposinf(loss).all())
    assert bool(L.linear_cross_entropy(x, w, torch.full_like(t, 5), high).isnan().all())
    nan = b.clone()
    nan[V - 1] = math.nan
    loss, lse = L.linear_cross_entropy(x, w, t, nan, save=True)
    assert bool(lse.isnan().all()) and bool(loss.isnan().all())


@pytest.mark.parametrize("dt", DTYPES)
def test_large_logits(dt):
    x, w, t, b, dloss = make(200, 1500, 256, dt, seed=9, scale=60.0)  # |z| of a few hundred
    _, lse = check_loss(x, w, t, b)
    check_grads(dloss, x, w, t, lse, b)


@pytest.mark.parametrize("dt", DTYPES)
def test_ignored_rows_count_for_nothing_whatever_they_hold(dt):
    M, V, K = 300, 900, 72
    x, w, t, b, dloss = make(M, V, K, dt, ignore=0.4, seed=10)
    lse = loss64(x, w, t, b)[2].float()
    clean = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
    loss = L.linear_cross_entropy(x, w, t, b)
    off = t == IGNORE
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(dt).min):
        y, e, d = x.clone(), lse.clone(), dloss.clone()
        y[off], e[off], d[off] = bad, bad, bad
        got = L.linear_cross_entropy_backward(d, y, w, t, e, b, need_db=True)
        assert all(torch.equal(p, q) for p, q in zip(got, clean)), bad
        assert torch.equal(L.linear_cross_entropy(y, w, t, b), loss), bad
        only = L.linear_cross_entropy_backward(d, y, w, t, e, b, need_dw=False)[0]
        assert bool((only[off] == 0).all()) and not bool(only.isnan().any()), bad
    nothing = torch.full_like(t, IGNORE)
    got = L.linear_cross_entropy_backward(dloss, x, w, nothing, lse, b, need_db=True)
    assert all(bool((g == 0).all()) for g in got)
    assert bool((L.linear_cross_entropy(x, w, nothing, b) == 0).all())


def test_another_ignored_index_and_targets_outside():
    M, V, K = 150, 333, 40
    x, w, t, b, dloss = make(M, V, K, torch.float16, ignore=0, seed=11)
    t[3], t[7], t[9] = 17, V, -100
    loss, lse = L.linear_cross_entropy(x, w, t, b, ignore_index=17, save=True)
    out = (t == V) | (t == -100)
    assert bool(loss[out].isnan().all()) and not bool(loss[~out].isnan().any()) and float(loss[3]) == 0.0
    assert not bool(lse.isnan().any())
    dx, _, _ = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, ignore_index=17, need_dw=False)
    assert bool(dx[out].isnan().all()) and not bool(dx[~out].isnan().any()) and bool((dx[3] == 0).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("K", [64, 65, 68])
def test_strides_and_alignments(K, dt):
    M, V = 150, 777
    x, w, t, b, dloss = make(M, V, K, dt, seed=12)
    loss, lse = check_loss(x, w, t, b)
    want = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
    for pad, off in ((8, 8), (3, 1), (1, 2)):
        big = torch.full((M, K + pad + off), math.nan, dtype=dt, device=DEV)
        y = big[:, off:off + K]
        y.copy_(x)
        flat = torch.empty(V * K + 9, dtype=dt, device=DEV)
        v = flat[off:off + V * K].view(V, K)
        v.copy_(w)
        bias = torch.empty(V + 9, dtype=dt, device=DEV)[off:off + V].copy_(b)
        assert torch.equal(L.linear_cross_entropy(y, v, t, bias), loss)
        got = L.linear_cross_entropy_backward(dloss, y, v, t, lse, bias, need_db=True)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    row = torch.empty(1, 2 * K, dtype=dt, device=DEV)[:, 1:1 + K].copy_(x[:1])
    assert torch.equal(L.linear_cross_entropy(row, w, t[:1], b), L.linear_cross_entropy(x[:1].clone(), w, t[:1], b))


@pytest.mark.parametrize("dt", DTYPES)
def test_no_columns_and_no_rows(dt):
    M, V = 37, 600
    x, w, t, b, dloss = make(M, V, 8, dt, seed=13)
    x0, w0 = x[:, :0].contiguous(), w[:, :0].contiguous()
    loss, lse = check_loss(x0, w0, t, b)
    plain, _ = L.linear_cross_entropy(x0, w0, t, save=True)
    assert float((plain[t != IGNORE] - math.log(V)).abs().max()) <= 2.0 ** -20
    dx, dw, db = L.linear_cross_entropy_backward(dloss, x0, w0, t, lse, b, need_db=True)
    assert dx.shape == (M, 0) and dw.shape == (V, 0)
    ref, e = grads64(dloss, x * 0, w, t, lse, b)[2]
    check(db, ref, e, "db")
    none = L.linear_cross_entropy(x[:0], w, t[:0], b)
    assert none.shape == (0,)
    dx, dw, db = L.linear_cross_entropy_backward(dloss[:0], x[:0], w, t[:0], lse[:0], b, need_db=True)
    assert dx.shape == (0, 8) and bool((dw == 0).all()) and bool((db == 0).all())


def test_nothing_is_written_outside_the_outputs():
    M, V, K = 131, 517, 67
    x, w, t, b, dloss = make(M, V, K, torch.float16, seed=14)
    band = 64
    bufs = {n: torch.full((s + 2 * band,), 77.0, dtype=d, device=DEV) for n, s, d in (
        ("loss", M, torch.float32), ("lse", M, torch.float32), ("dx", M * K, torch.float16),
        ("dw", V * K, torch.float16), ("db", V, torch.float16))}
    at = {n: v.data_ptr() + band * v.element_size() for n, v in bufs.items()}
    common = dict(x=x.data_ptr(), w=w.data_ptr(), b=b.data_ptr(), target=t.data_ptr(), M=M, V=V, K=K,
                  ignore_index=IGNORE, dtype=L.DTYPE_F16)
    s = torch.cuda.current_stream().cuda_stream
    assert L.poot_linear_cross_entropy(L.LinearCrossEntropyArgs(loss=at["loss"], lse=at["lse"], **common), s) == L.POOT_OK
    assert L.poot_linear_cross_entropy_backward(L.LinearCrossEntropyBackwardArgs(
        dloss=dloss.data_ptr(), dloss_stride=1, lse=at["lse"], dx=at["dx"], dw=at["dw"], db=at["db"], **common),
        s) == L.POOT_OK
    torch.cuda.synchronize()
    for n, v in bufs.items():
        assert bool((v[:band] == 77).all()) and bool((v[-band:] == 77).all()), n
    loss, lse = L.linear_cross_entropy(x, w, t, b, save=True)
    assert torch.equal(bufs["loss"][band:-band], loss) and torch.equal(bufs["lse"][band:-band], lse)
    assert L.poot_linear_device_status(0) == L.POOT_OK


def test_streams_and_graphs():
    """Two captured graphs and calls made outside them, on one stream and another."""
    sets = [make(260, 1100 + 64 * i, 128, torch.bfloat16, seed=15 + i) for i in range(2)]

    def step(s):
        x, w, t, b, dloss = s
        loss, lse = L.linear_cross_entropy(x, w, t, b, save=True)
        return (loss, *L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True))
    want = [step(s) for s in sets]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(s))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
        loose = step(sets[0])
    torch.cuda.synchronize()
    for got, ref in zip([*outs, loose], [*want, want[0]]):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
    # new inputs in the captured ones' place
    sets[0][0].neg_()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], step(sets[0])))
    x, w, t, b, _ = sets[1]
    side.wait_stream(torch.cuda.current_stream())
    loss = L.linear_cross_entropy(x, w, t, b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, want[1][0])


def test_refusals():
    x, w, t, b, dloss = make(8, 32, 16, torch.float16)
    lse = torch.zeros(8, device=DEV)
    for bad in (dict(x=x.float()), dict(w=w.bfloat16()), dict(target=t.int()), dict(bias=b.float())):
        with pytest.raises(TypeError):
            L.linear_cross_entropy(**{**dict(x=x, w=w, target=t, bias=b), **bad})
    for bad in (dict(x=x[0]), dict(x=x.t()), dict(w=w[:, :8]), dict(w=w.cpu()), dict(target=t[:4]), dict(bias=b[:3]),
                dict(target=torch.stack([t, t], 1)[:, 0])):
        with pytest.raises(ValueError):
            L.linear_cross_entropy(**{**dict(x=x, w=w, target=t, bias=b), **bad})
    good = dict(dloss=dloss, x=x, w=w, target=t, lse=lse, bias=b)
    for bad in (dict(dloss=dloss.double()), dict(lse=lse.half())):
        with pytest.raises(TypeError):
            L.linear_cross_entropy_backward(**{**good, **bad})
    for bad in (dict(dloss=dloss.sum()), dict(dloss=dloss[:3]), dict(lse=lse[:3]), dict(lse=lse.cpu())):
        with pytest.raises(ValueError):
            L.linear_cross_entropy_backward(**{**good, **bad})
    with pytest.raises(L.PootLinearError):
        L.linear_cross_entropy(x, w[:0], t)


def test_operands_beyond_2_to_the_31_elements():
    """Rows of x gigabytes apart; a W and its gradient whose last rows' offsets pass 32 bits."""
    x, w, t, b, dloss = make(1000, 300, 72, torch.float16, seed=21)
    big = torch.empty(1000 * 3_000_000, dtype=torch.float16, device=DEV)
    y = big.as_strided(x.shape, (3_000_000, 1)).copy_(x)
    loss, lse = L.linear_cross_entropy(x, w, t, b, save=True)
    assert torch.equal(L.linear_cross_entropy(y, w, t, b), loss)
    want = L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True)
    got = L.linear_cross_entropy_backward(dloss, y, w, t, lse, b, need_db=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    del big, y
    M, V, K = 5, 600_001, 4096
    g = torch.Generator(device=DEV).manual_seed(22)
    w = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, V, 100_000):
        w[i:i + 100_000] = torch.randn(min(100_000, V - i), K, generator=g, device=DEV) * 0.02
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    t = torch.tensor([0, V - 1, 524_287, 524_288, V - 2], device=DEV)
    _, lse = check_loss(x, w, t, None)
    check_grads(torch.rand(M, generator=g, device=DEV) + 0.5, x, w, t, lse, None, need_db=False)


def test_two_threads_on_one_stream():
    """Their calls share the stream's workspace, one call at a time."""
    sets = [make(200 + 90 * i, 1500, 70 + 8 * i, torch.float16, seed=23 + i) for i in range(2)]

    def step(s):
        x, w, t, b, dloss = s
        loss, lse = L.linear_cross_entropy(x, w, t, b, save=True)
        return (loss, *L.linear_cross_entropy_backward(dloss, x, w, t, lse, b, need_db=True))
    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        for _ in range(20):
            got[i].append(step(sets[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for out in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(out, want[i]))

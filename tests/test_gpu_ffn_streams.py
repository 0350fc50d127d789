"""The tensor calls, the linear's and the widened contraction's too, on a stream
that is not the current one: the caller may drop its tensors at once, and their
memory is not handed out again before that stream has read them."""
import pytest
import torch

import linear_fp16_gb300 as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _make(shapes, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).half().to(DEV) for s in shapes]


M, N, K = 384, 520, 264
CALLS = {
    "gated_linear": (((M, K), (N, K), (N, K), (N,), (N,)),
                     lambda t, s: L.gated_linear(*t, save=True, stream=s)),
    "gated_linear_decode": (((5, K), (N, K), (N, K), (N,), (N,)),
                            lambda t, s: [L.gated_linear(*t, stream=s)]),
    "gated_linear_backward": (((M, N), (M, K), (N, K), (N, K), (M, N), (M, N)),
                              lambda t, s: L.gated_linear_backward(*t, need_db=True, stream=s)),
    "linear": (((M, K), (N, K), (N,)), lambda t, s: [L.linear(*t, stream=s)]),
    "contract": (((M, K), (N, K), (N,), (M, N)),
                 lambda t, s: [L.contract(*t[:3], steps=["silu", ("mul", t[3])], stream=s)]),
    "linear_backward": (((M, N), (M, K), (N, K)), lambda t, s: L.linear_backward(*t, stream=s)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_inputs_dropped_after_the_call(name):
    shapes, call = CALLS[name]
    want = call(_make(shapes, 1), None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        warm = call(_make(shapes, 4), None)   # this stream's memory and workspace are there
    s.synchronize()
    del warm
    torch.full((4,), float("nan"), dtype=torch.float16, device=DEV)   # (loading a kernel waits for the device)
    tensors = _make(shapes, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)    # about 0.1 s before the call's first kernel
    got = call(tensors, s)
    where = {t.data_ptr() for t in tensors}
    sizes = [(t.shape, t.dtype) for t in tensors]
    del tensors
    again = [torch.full(sh, float("nan"), dtype=dt, device=DEV) for sh, dt in sizes]
    reused = where & {t.data_ptr() for t in again}
    assert not s.query()
    torch.cuda.synchronize()
    assert L.poot_linear_device_status(0) == L.POOT_OK
    assert not reused
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_and_results_of_a_clip_dropped_after_the_call():
    grads = _make(((3000,), (70, 90)), 2)
    want = float(L.clip_grad_norm(grads, 0.5, out=[torch.empty_like(g) for g in grads]))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.clip_grad_norm([torch.ones_like(g) for g in grads], 0.5)   # this stream's memory and workspace are there
    s.synchronize()
    out = [torch.empty_like(g) for g in grads]
    where = {t.data_ptr() for t in grads + out}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    norm = L.clip_grad_norm(grads, 0.5, out=out, stream=s)
    sizes = [(t.shape, t.dtype) for t in grads + out]
    del grads, out
    again = [torch.full(sh, float("nan"), dtype=dt, device=DEV) for sh, dt in sizes]
    reused = where & {t.data_ptr() for t in again}
    assert not s.query()
    torch.cuda.synchronize()
    assert not reused and float(norm) == want
    assert all(torch.isnan(t).all() for t in again)      # the clip wrote into nobody else's memory


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        stream_id, device_index, device_type = 0, 1, 1
    t = _make(((4, 8), (16, 8), (16, 8)), 3)
    with pytest.raises(ValueError):
        L.gated_linear(*t, stream=Elsewhere())
    with pytest.raises(ValueError):
        L.clip_grad_norm(t, 1.0, stream=Elsewhere())
    Elsewhere.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        L.linear(t[0], t[1], t[1][:, 0].contiguous(), stream=Elsewhere())


def test_a_stream_given_by_its_handle_alone():
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream
    x, w, b = _make(((40, 64), (48, 64), (48,)), 4)
    want = L.linear(x, w, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = L.linear(x, w, b, stream=Handle(s))
    s.synchronize()
    assert torch.equal(got, want)

"""The per-stream workspace under several host threads.

On the CPU: csrc/host.cuh with the CUDA runtime's functions replaced
(workspace_lease.cpp).  On a GPU: calls of two threads on one stream give the
bits of the same calls made alone.
"""
import os
import subprocess
import threading

import pytest
import torch

import linear_fp16_gb300 as L
from linear_fp16_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
DEV = "cuda:0"


def test_a_workspace_belongs_to_one_call_at_a_time(tmp_path):
    exe = str(tmp_path / "workspace_lease")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I", B.CSRC, "-I", B.INCLUDE, "-I", cuda,
                    os.path.join(HERE, "workspace_lease.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def _calls():
    """(name, call): operators that write their workspace with one launch and
    read it with another, each with inputs of its own."""
    g = torch.Generator().manual_seed(31)
    n = lambda *s: torch.randn(s, generator=g)
    h = lambda *s: n(*s).half().to(DEV)
    out = []
    for i in range(2):
        M, N, K = 96 + 40 * i, 264, 200
        bwd = (h(M, N), h(M, K), h(N, K), h(N, K), h(M, N), h(M, N))
        out.append((f"gated_linear_backward {i}",
                    lambda a=bwd: L.gated_linear_backward(*a, need_db=True)))
        odd = (h(M, 130), h(77, 130), h(77, 130))
        out.append((f"gated_linear, odd rows {i}", lambda a=odd: (L.gated_linear(*a),)))
        lin = (h(M, 130), h(77, 130), h(77))
        out.append((f"linear, odd rows {i}", lambda a=lin: (L.linear(*a),)))
        split = (h(64, 8192), h(512, 8192), h(512))
        out.append((f"linear, split {i}", lambda a=split: (L.linear(*a),)))
        noalloc = (h(64, 4096), h(512, 4096), h(512))

        def fixed(a=noalloc):
            y = torch.empty(64, 512, dtype=torch.float16, device=DEV)
            rc = L.poot_linear_f16_splitk_noalloc(a[0].data_ptr(), a[1].data_ptr(), a[2].data_ptr(), y.data_ptr(),
                                                  64, 512, 4096, 4, torch.cuda.current_stream().cuda_stream)
            assert rc == L.POOT_OK
            return (y,)
        out.append((f"linear, split in the fixed array {i}", fixed))
        grads = [n(5000 + 999 * i).to(DEV), h(300 + i)]

        def clip(gs=grads):
            o = [torch.empty_like(t) for t in gs]
            return (L.clip_grad_norm(gs, 0.5, out=o), *o)
        out.append((f"clip_grad_norm {i}", clip))
    return out


@pytest.mark.gpu
def test_two_host_threads_on_one_stream():
    calls = _calls()
    alone = [call() for _, call in calls]
    torch.cuda.synchronize()
    wrong, errors = [], []
    start = threading.Barrier(2)

    def work(i):
        try:
            torch.cuda.set_device(0)
            start.wait()
            for rep in range(60):
                results = [(k, calls[k][1]()) for k in range(len(calls)) if calls[k][0].endswith(str(i)) for _ in range(3)]
                for k, got in results:
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[k]) if a is not None):
                        wrong.append((rep, calls[k][0]))
        except Exception as e:  # reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert not wrong, wrong[:10]
    assert L.poot_linear_device_status(0) == L.POOT_OK

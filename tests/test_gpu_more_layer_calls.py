"""The layer norm, the 4-bit product and the gradients' norm as programs call them at once: host threads on one
stream, a stream's first call inside a capture, a norm in C without its optional results."""
import threading

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def test_host_threads_share_a_stream():
    """Calls that take the stream's workspace and grow it, from four threads: each as if it were alone."""
    stream = torch.cuda.Stream()
    jobs = []
    for k, (M, N) in enumerate(((300, 1000), (3000, 4096), (700, 16384), (900, 24000))):
        h, dy, w = randn((M, N), torch.bfloat16, 1 + k), randn((M, N), torch.bfloat16, 11 + k), randn(N, torch.bfloat16, 21 + k)
        grads = [randn(1_000_000 * (k + 1) + 7, torch.float32, 31 + k), randn(1001, torch.bfloat16, 41 + k)]
        fwd = mbt.tile_layernorm(h, w)
        want = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w)
        jobs.append((dy, h, fwd, w, grads, want, mbt.tile_grad_norm(grads, max_norm=1.0)))
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        torch.cuda.set_device(0)
        dy, h, fwd, w, grads, want, total = jobs[k]
        kept = []
        for _ in range(12):
            got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, stream=stream)
            norm = mbt.tile_grad_norm(grads, max_norm=1.0, stream=stream)
            kept.append((got, norm))
        stream.synchronize()
        for got, norm in kept:
            if not all(torch.equal(a, b) for a, b in zip(got, want)) or not torch.equal(norm.norm, total.norm):
                wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert mbt.tile_status()[0] == 0


def test_first_call_inside_a_capture():
    """Without the stream's workspace a captured call is refused and the capture lives on; calls that need none work."""
    big, few = [torch.ones(4_000_000, device="cuda")], [torch.ones(100, device="cuda")]
    x, w = randn((64, 512), torch.bfloat16, 51), randn((200, 512), torch.bfloat16, 52)
    fwd = mbt.tile_layernorm(x)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    refused = []
    with torch.cuda.graph(graph, stream=stream):
        for call in (lambda: mbt.tile_grad_norm(big),
                     lambda: mbt.tile_layernorm_backward(x, x, fwd.mean, fwd.rstd, None, dbias=torch.zeros(512, device="cuda"))):
            try:
                call()
            except mbt.MbtError as e:
                refused.append(e.code)
        got = mbt.tile_clip_grads(few, 5.0, eps=0.0)
        y = mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(mbt.tile_layernorm(x).out), mbt.tile_mx4_quantize(w))
    assert refused == [-8, -8]
    graph.replay()
    torch.cuda.synchronize()
    assert got.norm.item() == 10 and got.scale.item() == 0.5 and bool((few[0] == 0.5).all())
    assert torch.equal(y, mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(fwd.out), mbt.tile_mx4_quantize(w)))


@pytest.mark.parametrize("M,N,ld", [(3, 100, 100), (3, 100, 103), (2000, 4096, 4096), (2000, 1001, 1001), (2, 70000, 70000)])
def test_a_residual_without_its_sum(M, N, ld):
    """residual given, residual_out not: the norm of the sum, nothing written beside it."""
    x, r = (torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")[:, :N] for _ in range(2))
    x.copy_(randn((M, N), torch.bfloat16, 61))
    r.copy_(randn((M, N), torch.bfloat16, 62))
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    rc = mbt.C.tile_layernorm(x.data_ptr(), r.data_ptr(), None, None, out.data_ptr(), None, None, mean.data_ptr(), rstd.data_ptr(),
                              M, N, ld, ld, 0, 0, 1, 0, -1, 1e-5, 0.0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want = mbt.tile_layernorm(x, residual=r)
    assert torch.equal(out, want.out) and torch.equal(mean, want.mean) and torch.equal(rstd, want.rstd)


def test_norms_without_a_factor():
    """scale NULL in C: the norm alone; max_norm infinity: the factor is grad_scale."""
    for n in (1000, 3_000_001):
        g = randn(n, torch.float32, 71)
        norm = torch.zeros(1, device="cuda")

        class Grad(mbt.layer.ctypes.Structure):
            _fields_ = [("p", mbt.layer.ctypes.c_void_p), ("n", mbt.layer.ctypes.c_int64), ("d", mbt.layer.ctypes.c_int32),
                        ("r", mbt.layer.ctypes.c_int32)]

        t = Grad(g.data_ptr(), n, 2, 0)
        rc = mbt.C.tile_grad_norm(mbt.layer.ctypes.byref(t), 1, None, 1.0, 1e-6, norm.data_ptr(), None,
                                  torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(norm[0], mbt.tile_grad_norm([g]).norm)

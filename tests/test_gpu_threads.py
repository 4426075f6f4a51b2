"""Host threads that share a stream, and with it the library's workspace."""
import threading

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import randn

pytestmark = pytest.mark.gpu
BF16, F32 = mbt.DTYPE_CODE[torch.bfloat16], mbt.DTYPE_CODE[torch.float32]


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def product(T, N, K, seed):
    """(call on a stream, out, expected): a 4-bit product that takes three kernels."""
    x = randn((T, K), torch.bfloat16, seed)
    q = torch.randint(0, 256, (N, K // 2), generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=torch.uint8)
    s = torch.full((N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    out, want = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"), mbt.tile_w4_matvec(x, q, s)

    def call(st):
        return mbt.C.tile_w4_matvec(x.data_ptr(), None, q.data_ptr(), s.data_ptr(), None, out.data_ptr(), T, N, K, 0, 0,
                                    0, 128, 0, BF16, BF16, BF16, st)

    return call, out, want, (x, q, s)


def gradient(M, N, seed):
    """The same of a norm's gradient with dweight: two kernels."""
    h, dy, w = (randn(k, torch.bfloat16, seed + i) for i, k in enumerate(((M, N), (M, N), N)))
    rstd = mbt.tile_rmsnorm(h, w).rstd
    dx, want = mbt.tile_rmsnorm_backward(dy, h, rstd, w)
    dw = torch.zeros_like(want)

    def call(st):
        return mbt.C.tile_rmsnorm_backward(dy.data_ptr(), h.data_ptr(), rstd.data_ptr(), w.data_ptr(), None, dx.data_ptr(),
                                           dw.data_ptr(), M, N, 0, 0, 0, 0, BF16, BF16, 0.0, st)

    return call, dw, want, (h, dy, w, rstd, dx)


def row_sum(M, N, seed):
    """The same of a row sum whose bands are split over CTAs: one kernel, tickets."""
    x = randn((M, N), torch.float32, seed)
    want = mbt.tile_rowsum(x, None, 64, 128, 3)
    out = torch.zeros_like(want)

    def call(st):
        return mbt.C.tile_rowsum(x.data_ptr(), out.data_ptr(), M, N, 64, 128, 3, F32, st)

    return call, out, want, (x,)


@pytest.mark.parametrize("grow", [False, True])
def test_calls_of_threads_on_one_stream(grow):
    """Every thread's results are those it gets alone; with `grow` the workspace starts small and grows under way."""
    work = [product(8, 512, 4096, 1), product(8, 768, 8192, 2), gradient(700, 2048, 3), row_sum(300, 40960, 6),
            gradient(1000, 5000, 7), product(5, 1000, 2048, 10)]
    torch.cuda.synchronize()
    stream, codes, right = torch.cuda.Stream(), [], [True] * len(work)
    if not grow:
        for call, *_ in work:
            assert call(stream.cuda_stream) == 0
    start = threading.Barrier(len(work))

    def run(k):
        torch.cuda.set_device(0)
        call, out, want, _ = work[k]
        mine = torch.cuda.Stream()
        start.wait()
        for _ in range(20):
            for _ in range(10):
                codes.append(call(stream.cuda_stream))   # (ctypes lets the other threads run meanwhile)
            done = torch.cuda.Event()
            done.record(stream)
            done.synchronize()
            with torch.cuda.stream(mine):
                right[k] = right[k] and torch.equal(out, want)

    for rep in range(3):
        if grow:
            mbt.tile_workspace_release(stream)
        threads = [threading.Thread(target=run, args=(k,)) for k in range(len(work))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    assert set(codes) == {0} and len(codes) == 3 * 200 * len(work)
    assert all(right)
    assert mbt.tile_status()[0] == 0
    mbt.tile_workspace_release(stream)


def test_graphs_outlive_the_growth_of_the_workspace():
    """A captured product and gradient are replayed after larger calls on their stream, and others on other streams."""
    small = [product(8, 512, 4096, 20), gradient(500, 1024, 21)]
    large = product(8, 4096, 16384, 24)
    others = [product(8, 512, 4096, 25 + k) for k in range(6)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for call, *_ in small:
        assert call(stream.cuda_stream) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        codes = [call(stream.cuda_stream) for call, *_ in small]
    assert codes == [0, 0]
    assert large[0](stream.cuda_stream) == 0
    stream.synchronize()
    streams = [torch.cuda.Stream() for _ in others]
    for _ in range(20):
        for (call, *_), st in zip(others, streams):
            assert call(st.cuda_stream) == 0
        for _, out, *_ in small:
            out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        for (call, *_), st in zip(others, streams):
            assert call(st.cuda_stream) == 0
        torch.cuda.synchronize()
        for _, out, want, _ in (*small, large, *others):
            assert torch.equal(out, want)
    del graph
    for st in (stream, *streams):
        mbt.tile_workspace_release(st)
    assert mbt.tile_status()[0] == 0

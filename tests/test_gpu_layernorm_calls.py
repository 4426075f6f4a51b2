"""tile_layernorm where outputs overwrite inputs crosswise, and in graphs replayed one after the other."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import TYPES, pitched, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("M,N,pad", [(5, 1000, 0), (65, 1001, 3), (3, 70000, 0), (2600, 4001, 0), (2600, 4096, 8), (700, 16384, 0),
                                     (400, 20001, 0), (311, 12001, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_out_over_the_residual_and_the_sum_over_x(M, N, pad, dtype):
    dt = TYPES[dtype]
    x, r = (pitched(randn((M, N), dt, seed), pad) for seed in (1, 2))
    w, b = randn(N, dt, 3), randn(N, dt, 4)
    want = mbt.tile_layernorm(x, w, b, r, out=torch.empty_strided(x.shape, x.stride(), dtype=dt, device="cuda"),
                              residual_out=torch.empty_strided(x.shape, x.stride(), dtype=dt, device="cuda"))
    got = mbt.tile_layernorm(x, w, b, r, out=r, residual_out=x)
    for p, q in zip((r, x, got.mean, got.rstd), (want.out, want.residual, want.mean, want.rstd)):
        assert torch.equal(p, q)
    assert mbt.tile_status()[0] == 0


def test_two_graphs_of_one_stream():
    """Graphs captured on one stream share its workspace; replayed in turn each gives its own gradients."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sets = []
    for M, N, seed in ((1500, 4096, 10), (40, 24576, 20)):
        h, dy, w = randn((M, N), torch.bfloat16, seed), randn((M, N), torch.bfloat16, seed + 1), randn(N, torch.bfloat16, seed + 2)
        fwd = mbt.tile_layernorm(h, w)
        want = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w)
        sets.append((h, dy, w, fwd, want))
    s.wait_stream(torch.cuda.current_stream())
    for h, dy, w, fwd, _ in sets:                      # (the workspace grows outside of a capture)
        mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, stream=s)
    s.synchronize()
    graphs = []
    for h, dy, w, fwd, want in sets:
        out = [torch.zeros_like(t) for t in want]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, dx=out[0], dweight=out[1], dbias=out[2])
        graphs.append((g, out, want))
    for _ in range(3):
        for g, out, _ in graphs:
            for t in out:
                t.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out, want in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert mbt.tile_status()[0] == 0

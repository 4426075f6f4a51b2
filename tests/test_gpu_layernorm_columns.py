"""tile_layernorm_backward's dweight and dbias where every sum is exact: each row counts once.

dy, h and mean are small integers and rstd a power of two from 1/2 to 2, so that dy xh is a
multiple of 1/2 of at most 2 * 4 * 2 = 16 and a column's sums stay below 2^24 halves for
M <= 2^19: fp32 holds every partial sum, in any order, and the results have to be equal."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import TYPES, gen, pitched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def integers(shape, most, seed):
    return torch.randint(-most, most + 1, shape, generator=gen(seed), device="cuda")


def check(M, N, dt, pad=0, offset=0, dres=False, one=None):
    dy, h = (pitched(integers((M, N), most, seed).to(dt), pad, offset) for most, seed in ((2, 1), (3, 2)))
    mean = integers((M,), 1, 3).float()
    rstd = torch.exp2(integers((M,), 1, 4).float())
    w = torch.ones(N, dtype=dt, device="cuda")
    r = pitched(integers((M, N), 1, 5).to(dt), pad, offset) if dres else None
    given = {}
    if one:                                            # only this one of the two
        w, given = None, {one: torch.empty(N, device="cuda")}
    dx, dw, db = mbt.tile_layernorm_backward(dy, h, mean, rstd, w, dresidual=r, **given)
    assert (dw is None) == (one == "dbias") and (db is None) == (one == "dweight")
    if dw is not None:
        assert torch.equal(dw.double(), (dy.double() * (h.double() - mean.double()[:, None]) * rstd.double()[:, None]).sum(0))
    if db is not None:
        assert torch.equal(db.double(), dy.double().sum(0))
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", [(1, 1), (1, 4096), (2, 7), (33, 1024), (151, 4096), (153, 4096), (305, 8192), (593, 4280),
                                 (700, 16384), (2100, 5001), (9001, 1032), (2047, 5001), (30001, 100), (50001, 24), (65537, 128),
                                 (40001, 16), (131073, 8)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_every_row_counts(M, N, dtype, dres):
    check(M, N, TYPES[dtype], dres=dres)


@pytest.mark.parametrize("M,N,pad,offset", [(301, 24576, 0, 0), (1000, 24000, 0, 0), (303, 20001, 7, 0), (41, 32768, 0, 0),
                                            (2049, 1001, 3, 1), (77, 512, 0, 1), (129, 12000, 8, 0), (65, 70001, 0, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_past_the_ring(M, N, pad, offset, dtype):
    """Rows too long, or that start anywhere: by chunks and by elements."""
    check(M, N, TYPES[dtype], pad, offset, dres=M % 2 == 0)


@pytest.mark.parametrize("one", ["dweight", "dbias"])
@pytest.mark.parametrize("M,N", [(305, 8192), (301, 24576)])
def test_one_of_the_two(one, M, N):
    check(M, N, torch.bfloat16, one=one)

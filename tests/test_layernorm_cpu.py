"""tile_layernorm and its gradient without a GPU: argument errors."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from mbarrier_async_tile_gb300 import _build

A, B, C_, D = 0x10000, 0x20000, 0x30000, 0x40000   # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_library():
    _build.build()


def norm(x=A, res=0, w=B, b=B, out=C_, ro=0, scales=0, mean=D, rstd=D, M=4, N=64, ld=(0, 0, 0, 0), dt=0, wdt=0, quant=-1,
         eps=1e-6):
    return mbt.C.tile_layernorm(x, res, w, b, out, ro, scales, mean, rstd, M, N, *ld, dt, wdt, quant, eps, 0.0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=0), -1), (dict(out=0), -1), (dict(mean=0), -1), (dict(rstd=0), -1), (dict(M=-1), -1), (dict(N=-1), -1),
    (dict(dt=3), -1), (dict(wdt=3), -1), (dict(w=0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(quant=16), -3), (dict(quant=0), -1), (dict(scales=A), -1), (dict(ro=A), -1), (dict(ld=(63, 0, 0, 0)), -1),
    (dict(ld=(0, 0, 1, 0)), -1), (dict(x=A + 1), -2), (dict(mean=D + 2), -2), (dict(rstd=D + 2), -2), (dict(w=B + 1), -2),
    (dict(b=B + 1), -2), (dict(M=1 << 40, N=1 << 30), -1),
])
def test_argument_errors(bad, code):
    assert norm(**bad) == code


def test_no_rows():
    assert norm(M=0, x=0, out=0, mean=0, rstd=0) == 0


def grad(dy=A, h=B, mean=C_, rstd=C_, w=D, dres=0, dx=A, dw=D, db=D, M=4, N=64, ld=(0, 0, 0, 0), dt=1, wdt=1):
    return mbt.C.tile_layernorm_backward(dy, h, mean, rstd, w, dres, dx, dw, db, M, N, *ld, dt, wdt, 0.0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dy=0), -1), (dict(h=0), -1), (dict(mean=0), -1), (dict(rstd=0), -1), (dict(dx=0), -1), (dict(M=-1), -1),
    (dict(dt=3), -1), (dict(ld=(0, 5, 0, 0)), -1), (dict(dx=A + 1), -2), (dict(dw=D + 2), -2), (dict(db=D + 2), -2),
    (dict(mean=C_ + 1), -2), (dict(rstd=C_ + 1), -2),
])
def test_gradient_argument_errors(bad, code):
    assert grad(**bad) == code
    assert grad(N=0) == 0


def test_python_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="quant"):
        mbt.tile_layernorm(x, quant=16)
    with pytest.raises(ValueError, match="CUDA"):
        mbt.tile_layernorm(x)
    with pytest.raises(ValueError, match="CUDA"):
        mbt.tile_layernorm_backward(x, x, x, x)

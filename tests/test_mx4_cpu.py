"""Microscaled 4-bit floats without a GPU: refusals, the scales' size, the tests' own reading of the formats."""
import itertools

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from mbarrier_async_tile_gb300 import _build
from mx4_helpers import E2M1, codes_of, nearest_code, quantise, tile_scales, untile_scales, values64

A, B, C_, D = 0x10000, 0x20000, 0x30000, 0x40000   # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_library():
    _build.build()


def quantize(x=A, ts=0, q=B, s=C_, M=4, K=64, ld=(0, 0), block=16, dt=1):
    return mbt.C.tile_mx4_quantize(x, ts, q, s, M, K, *ld, block, dt, None)


def dequantize(q=B, s=C_, ts=0, out=A, M=4, K=64, ld=(0, 0), block=16, dt=1):
    return mbt.C.tile_mx4_dequantize(q, s, ts, out, M, K, *ld, block, dt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=0), -1), (dict(s=0), -1), (dict(M=-1), -1), (dict(K=-32), -1), (dict(dt=3), -1), (dict(K=48), -3),
    (dict(block=64), -3), (dict(block=32, ts=A), -1), (dict(q=B + 8), -2), (dict(s=C_ + 8), -2), (dict(ts=D + 2), -2),
])
def test_conversion_argument_errors(bad, code):
    assert quantize(**bad) == code
    assert dequantize(**bad) == code


def test_conversion_pitches_and_nothing():
    assert quantize(x=0) == -1 and dequantize(out=0) == -1
    assert quantize(x=A + 1) == -2 and dequantize(out=A + 1) == -2
    assert quantize(ld=(63, 0)) == -1 and quantize(ld=(0, 16)) == -1 and quantize(ld=(0, 40)) == -2
    assert dequantize(ld=(16, 0)) == -1 and dequantize(ld=(0, 63)) == -1 and dequantize(ld=(40, 0)) == -2
    assert quantize(M=0, x=0, q=0, s=0) == 0 and quantize(K=0) == 0 and dequantize(M=0) == 0


def matmul(a=A, sa=B, ta=0, b=C_, sb=D, tb=0, out=A, M=4, N=8, K=64, ld=(0, 0, 0), block=16, odt=1):
    return mbt.C.tile_mx4_matmul(a, sa, ta, b, sb, tb, out, M, N, K, *ld, block, odt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(a=0), -1), (dict(sa=0), -1), (dict(b=0), -1), (dict(sb=0), -1), (dict(out=0), -1), (dict(M=-1), -1),
    (dict(N=-1), -1), (dict(K=1 << 31), -1), (dict(odt=3), -1), (dict(K=80), -3), (dict(block=128), -3),
    (dict(block=32, tb=A), -1), (dict(ld=(16, 0, 0)), -1), (dict(ld=(0, 40, 0)), -2), (dict(ld=(0, 0, 7)), -1),
    (dict(a=A + 4), -2), (dict(sb=D + 4), -2), (dict(out=A + 1), -2), (dict(ta=A + 2), -2),
])
def test_product_argument_errors(bad, code):
    assert matmul(**bad) == code
    assert matmul(M=0) == 0 and matmul(N=0) == 0


def test_scale_bytes():
    for M, K, block in itertools.product((0, 1, 128, 129), (0, 32, 64, 96, 4096), (16, 32)):
        want = -(-M // 128) * -(-(K // block) // 4) * 512
        assert mbt.C.tile_mx4_scale_bytes(M, K, block) == want
    assert mbt.C.tile_mx4_scale_bytes(1, 32, 8) == -1 and mbt.C.tile_mx4_scale_bytes(-1, 32, 16) == -1


def test_reading_of_the_formats():
    """Every code's value is its own code; halfway values go to the even one; the tiles hold each byte once."""
    v = torch.tensor(E2M1 + [-x for x in E2M1])
    assert nearest_code(v).tolist() == list(range(16))
    half = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])])
    assert nearest_code(half).tolist() == [0, 2, 2, 4, 4, 6, 6]
    b = torch.randint(0, 256, (300, 13), dtype=torch.uint8)
    tiles = tile_scales(b)
    assert tiles.shape == (3, 4, 512) and torch.equal(untile_scales(tiles, 300, 13), b)
    assert int((tiles != 0).sum()) == int((b != 0).sum())
    x = torch.tensor([[1.0, -6.0, 0.25, 0.0] * 8])
    for block in (16, 32):
        q, s = quantise(x, block)
        assert torch.equal(values64(q, s, block).float()[:, :4], torch.tensor([[1.0, -6.0, 0.0, 0.0]]))
        assert codes_of(q).shape == x.shape


def test_python_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="block"):
        mbt.tile_mx4_quantize(x, block=8)
    m = mbt.Mx4(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="one size"):
        mbt.tile_mx4_matmul(m, m._replace(block=32))
    with pytest.raises(ValueError, match="output type"):
        mbt.tile_mx4_dequantize(m, dtype=torch.int8)
    with pytest.raises(ValueError, match="Mx4"):
        mbt.tile_mx4_matmul((m.q, m.scales), m)
    for call in (lambda: mbt.tile_mx4_quantize(x), lambda: mbt.tile_mx4_dequantize(m), lambda: mbt.tile_mx4_matmul(m, m)):
        with pytest.raises(ValueError, match="CUDA"):
            call()

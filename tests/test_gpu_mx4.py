"""Microscaled 4-bit floats: quantisation code by code, the product against the formula in 64 bits.

Product: an instruction adds 64 products to a sum in fp32.  Whatever the order and the
rounding within it (to nearest, or cut off), it is off by at most 4 u of the magnitudes that
it adds, and a result goes through K / 64 of them and a few more additions:
4 u (K / 64 + 8) sum |a| |b| and the output's rounding bound it."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import OUT_U, TINY, TYPES, U, gen, randn, worst
from mx4_helpers import quantise, scale64, tile_scales, untile_scales, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def check_quantised(x, block, ts, m):
    M, K = x.shape
    q, s = quantise(x, block, ts)
    assert m.q.shape == (M, K // 2) and m.block == block and m.tensor_scale is ts
    assert torch.equal(m.scales, tile_scales(s))
    assert torch.equal(m.q & 0x77, q & 0x77)                 # magnitudes; signs where there is something to sign
    some = torch.stack((q & 7, q >> 4 & 7), 2) > 0
    sign = torch.stack((m.q ^ q, (m.q ^ q) >> 4), 2) & 8
    assert not bool((sign.bool() & some).any())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 8192), (3, 96), (33, 64), (128, 256), (129, 1056), (300, 480), (1000, 2080)])
def test_quantise(M, K, dtype, block):
    x = randn((M, K), TYPES[dtype], 1, 3.0)
    x[M // 2, :32] = 0
    ts = None if block == 32 or K % 64 else (x.abs().amax().float() / 2688).view(1)
    m = mbt.tile_mx4_quantize(x, block=block, tensor_scale=ts)
    check_quantised(x, block, ts, m)
    for out in TYPES.values():
        s = untile_scales(m.scales, M, K // block)
        t = ts if ts is not None else torch.ones(1, device="cuda")
        want = (values64(m.q, s, block).float() * t).to(out)   # (code times scale is exact in fp32)
        assert torch.equal(mbt.tile_mx4_dequantize(m, dtype=out), want)


@pytest.mark.parametrize("block", [16, 32])
def test_quantise_halves_and_extremes(block):
    """Values on and next to every border, of blocks of every size that fp32 holds."""
    base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda")
    near = torch.stack((base.nextafter(base * 0), base, base.nextafter(base * 2), -base), 1).flatten()   # 32 values
    near[3] = 6.0
    e = torch.arange(-100 if block == 16 else -149, 40 if block == 16 else 125, device="cuda").double()
    x = (near.double() * 2.0 ** e[:, None]).float().repeat(1, 2)
    check_quantised(x, block, None, mbt.tile_mx4_quantize(x, block=block))
    if block == 16:
        for t in (2.0 ** -60, 0.0123, 3.3e7, 2.0 ** 60):
            ts = torch.full((1,), t, device="cuda")
            check_quantised(x, block, ts, mbt.tile_mx4_quantize(x, block=block, tensor_scale=ts))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_blocks_that_are_not_finite(block, bad):
    x = randn((5, 128), torch.float32, 3)
    x[2, 70] = bad
    m = mbt.tile_mx4_quantize(x, block=block)
    check_quantised(x, block, None, m)
    v = mbt.tile_mx4_dequantize(m, dtype=torch.float32)
    where = torch.zeros(5, 128, dtype=torch.bool, device="cuda")
    where[2, 70 // block * block:(70 // block + 1) * block] = True
    assert torch.equal(v.isnan(), where)
    b = mbt.tile_mx4_quantize(randn((40, 128), torch.float32, 4), block=block)
    for M in (5, 200):                                        # few rows, many
        a = mbt.tile_mx4_quantize(x.repeat(M // 5, 1), block=block)
        y = mbt.tile_mx4_matmul(a, b)
        rows = torch.arange(M, device="cuda") % 5 == 2
        assert torch.equal(y.isnan(), rows[:, None].expand(M, 40))


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_quantise_pitches(pad, offset):
    store = torch.full((70 * (96 + pad) + offset,), float("nan"), device="cuda", dtype=torch.bfloat16)
    x = store[offset:].view(70, 96 + pad)[:, :96]
    x.copy_(randn((70, 96), torch.bfloat16, 5))
    wide = torch.full((70, 80), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 2, 512), 0x55, dtype=torch.uint8, device="cuda")
    m = mbt.tile_mx4_quantize(x, q=wide[:, 16:64], scales=scales)
    check_quantised(x, 16, None, m)
    assert bool((wide[:, :16] == 0x55).all()) and bool((wide[:, 64:] == 0x55).all())
    out = torch.full((70 * (96 + pad) + offset,), 7.0, device="cuda", dtype=torch.bfloat16)
    view = out[offset:].view(70, 96 + pad)[:, :96]
    mbt.tile_mx4_dequantize(m, out=view)
    assert torch.equal(view, mbt.tile_mx4_dequantize(m)) and bool((out[:offset] == 7).all())
    assert bool((out[offset:].view(70, 96 + pad)[:, 96:] == 7).all())


def operand(M, K, block, seed, ts=None, pitch=0, fill=0):
    """Any codes and scales, in rows `pitch` bytes longer."""
    g = gen(seed)
    store = torch.randint(0, 256, (M, K // 2 + pitch), generator=g, device="cuda", dtype=torch.uint8)
    low, high = (0x20, 0x50) if block == 16 else (120, 135)
    s = torch.randint(low, high, (M, K // block), generator=g, device="cuda", dtype=torch.uint8)
    t = None if ts is None else torch.full((1,), ts, device="cuda")
    m = mbt.Mx4(store[:, :K // 2], tile_scales(s, fill), t, block)
    return m, values64(m.q, s, block, t)


def check_product(a, va, b, vb, got, K):
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    bound = 4 * U * (K / 64 + 8) * size + (OUT_U[got.dtype] + 2 * U) * want.abs() + TINY[got.dtype]
    assert worst(got, want, bound) <= 1


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K", [32, 64, 96, 256, 288, 1024, 4128])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 130), (2, 1000), (16, 128), (17, 7), (31, 300), (33, 129), (64, 64), (65, 257),
                                 (127, 500), (128, 128), (129, 40), (200, 129), (300, 1000)])
def test_product(M, N, K, block):
    t = 0.01 if block == 16 and K % 64 == 0 else None
    a, va = operand(M, K, block, 10, t)
    b, vb = operand(N, K, block, 11, t)
    check_product(a, va, b, vb, mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32), K)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M", [1, 20, 40, 100, 128, 129, 700])
@pytest.mark.parametrize("block", [16, 32])
def test_product_is_exact_where_sums_are(M, block):
    """Small multiples of one power of two, whose sums fit fp32: every bit, in every variant."""
    K, N = 1120, 333
    a, va = operand(M, K, block, 12)
    b, vb = operand(N, K, block, 13)
    one = torch.full((1, 1), 0x38 if block == 16 else 127, dtype=torch.uint8, device="cuda")
    two = torch.full((1, 1), 0x40 if block == 16 else 128, dtype=torch.uint8, device="cuda")
    sa = torch.where(torch.rand(M, K // block, generator=gen(14), device="cuda") < 0.5, one, two)
    sb = torch.where(torch.rand(N, K // block, generator=gen(15), device="cuda") < 0.5, one, two)
    a, b = a._replace(scales=tile_scales(sa)), b._replace(scales=tile_scales(sb))
    want = values64(a.q, sa, block) @ values64(b.q, sb, block).t()
    got = mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32)
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (8, 8191, 8160), (17, 640, 16384), (100, 20000, 512), (2047, 1000, 2048),
                                   (1000, 4096, 4096), (4100, 4100, 288)])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_product_large(M, N, K, out):
    a, va = operand(M, K, 16, 20, 2e-3)
    b, vb = operand(N, K, 16, 21, 2e-3)
    got = mbt.tile_mx4_matmul(a, b, out_dtype=TYPES[out])
    check_product(a, va, b, vb, got, K)
    assert torch.equal(got, mbt.tile_mx4_matmul(a, b, out_dtype=TYPES[out]))
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product_pitches(M, pad, offset, out):
    """Pitched codes and outputs; scale bytes of rows that are not there are NaN."""
    K, N = 320, 131
    a, va = operand(M, K, 16, 22, pitch=48)
    b, vb = operand(N, K, 16, 23, pitch=16)
    store = torch.full((M * (N + pad) + offset + 8,), 7.0, device="cuda", dtype=TYPES[out])
    view = store[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    got = mbt.tile_mx4_matmul(a, b, out=view)
    assert got.data_ptr() == view.data_ptr()
    check_product(a, va, b, vb, view, K)
    kept = torch.ones_like(store, dtype=torch.bool)
    kept[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N] = False
    assert bool((store[kept] == 7).all())


@pytest.mark.parametrize("M", [3, 150])
def test_scales_of_rows_that_are_not_there(M):
    K, N = 256, 100
    (a, va), (b, vb) = operand(M, K, 16, 24, fill=0x7F), operand(N, K, 16, 25, fill=0x7F)
    check_product(a, va, b, vb, mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32), K)


def test_empty_products():
    a, _ = operand(3, 64, 16, 26)
    z = a._replace(q=a.q[:, :0], scales=a.scales[:, :0])
    assert torch.equal(mbt.tile_mx4_matmul(z, z), torch.zeros(3, 3, device="cuda", dtype=torch.bfloat16))
    none = a._replace(q=a.q[:0], scales=a.scales[:0])
    assert mbt.tile_mx4_matmul(none, a).shape == (0, 3) and mbt.tile_mx4_matmul(a, none).shape == (3, 0)
    assert mbt.tile_mx4_quantize(torch.zeros(0, 64, device="cuda")).q.shape == (0, 32)
    assert mbt.tile_mx4_dequantize(none).shape == (0, 64)


def test_gpu_refusals():
    a, _ = operand(3, 64, 16, 27)
    for bad in (a._replace(scales=a.scales[:, :, :256]), a._replace(q=a.q.float()), a._replace(q=a.q[:, ::2]),
                a._replace(q=a.q[:, 8:24]), a._replace(tensor_scale=torch.ones(2, device="cuda")),
                a._replace(scales=a.scales.cpu()), a._replace(block=32, tensor_scale=torch.ones(1, device="cuda"))):
        with pytest.raises((ValueError, mbt.MbtError)):
            mbt.tile_mx4_matmul(bad, bad)
    with pytest.raises(ValueError):
        mbt.tile_mx4_matmul(a, operand(3, 128, 16, 28)[0])
    with pytest.raises(ValueError):
        mbt.tile_mx4_quantize(torch.zeros(3, 40, device="cuda"))
    with pytest.raises(ValueError):
        mbt.tile_mx4_matmul(a, a, out=torch.empty(3, 3, device="cuda"), out_dtype=torch.bfloat16)


def test_streams_and_graphs():
    """Quantise and multiply on another stream, captured and replayed with new values."""
    w = mbt.tile_mx4_quantize(randn((500, 512), torch.bfloat16, 30))
    x = randn((9, 512), torch.bfloat16, 31)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(x), w)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(x, stream=side), w, stream=side), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(x), w)
    x.copy_(randn((9, 512), torch.bfloat16, 32))
    graph.replay()
    assert torch.equal(y, mbt.tile_mx4_matmul(mbt.tile_mx4_quantize(x), w))


def test_written_tensors_raise_their_version():
    x = randn((9, 64), torch.bfloat16, 33)
    m = mbt.tile_mx4_quantize(x)
    out = torch.empty(9, 9, device="cuda", dtype=torch.bfloat16)
    before = out._version, m.q._version
    mbt.tile_mx4_matmul(m, m, out=out)
    mbt.tile_mx4_quantize(x, q=m.q, scales=m.scales)
    assert out._version > before[0] and m.q._version > before[1]
    assert scale64(m.scales[0, 0, :1], 16).isfinite().all()


# 256 x 256 tiles for every pair of SMs, with edges of every kind
PAIRS = [(2560, 2560), (2500, 2601), (257, 20001), (20001, 300), (2305, 2432), (4097, 2433)]


@pytest.mark.parametrize("M,N", PAIRS)
@pytest.mark.parametrize("K", [32, 96, 1024, 4128])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product_by_pairs(M, N, K, block, out):
    t = 0.03 if block == 16 else None
    a, va = operand(M, K, block, 40, t, pitch=16)
    b, vb = operand(N, K, block, 41, t, fill=0x7F if block == 16 and K % 64 == 0 else 0)
    got = mbt.tile_mx4_matmul(a, b, out_dtype=TYPES[out])
    check_product(a, va, b, vb, got, K)
    assert torch.equal(got, mbt.tile_mx4_matmul(a, b, out_dtype=TYPES[out]))
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("block", [16, 32])
def test_pairs_are_exact_where_sums_are(block):
    M, N, K = 2600, 2561, 1120
    a, va = operand(M, K, block, 42)
    b, vb = operand(N, K, block, 43)
    one, two = ((0x38, 0x40) if block == 16 else (127, 128))
    sa = torch.where(torch.rand(M, K // block, generator=gen(44), device="cuda") < 0.5, one, two).to(torch.uint8)
    sb = torch.where(torch.rand(N, K // block, generator=gen(45), device="cuda") < 0.5, one, two).to(torch.uint8)
    a, b = a._replace(scales=tile_scales(sa)), b._replace(scales=tile_scales(sb))
    want = values64(a.q, sa, block) @ values64(b.q, sb, block).t()
    assert torch.equal(mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_pairs_pitches(pad, offset, out):
    M, N, K = 2570, 2443, 320
    a, va = operand(M, K, 16, 46, 1e-3)
    b, vb = operand(N, K, 16, 47, 1e-2)
    store = torch.full((M * (N + pad) + offset + 8,), 7.0, device="cuda", dtype=TYPES[out])
    view = store[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    mbt.tile_mx4_matmul(a, b, out=view)
    check_product(a, va, b, vb, view, K)
    kept = torch.ones_like(store, dtype=torch.bool)
    kept[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N] = False
    assert bool((store[kept] == 7).all())


def test_past_four_gib():
    """Rows whose offsets pass 32 bits, of elements, codes and results."""
    M, K = 140001, 65536
    x = torch.ones(1, 1, dtype=torch.float16, device="cuda").expand(M, K).contiguous()
    x[-3:] = randn((3, K), torch.float16, 50)
    m = mbt.tile_mx4_quantize(x)
    assert m.q.numel() > 1 << 32
    last = mbt.tile_mx4_quantize(x[-3:])
    assert torch.equal(m.q[-3:], last.q)
    assert torch.equal(untile_scales(m.scales, M, K // 16)[-3:], untile_scales(last.scales, 3, K // 16))
    back = mbt.tile_mx4_dequantize(m, dtype=torch.float16, out=x)
    # (ones: 1 / 6 is 10.67 steps of 1 / 64, the scale 11 / 64, 1 by it 5.8, code 6: 66 / 64)
    assert torch.equal(back[-3:], mbt.tile_mx4_dequantize(last, dtype=torch.float16)) and bool((back[:5] == 66 / 64).all())
    del x, back
    few, many = operand(2, K, 16, 51)[0], operand(150, K, 16, 52)[0]
    want = mbt.tile_mx4_matmul(few, last, out_dtype=torch.float32)
    assert torch.equal(mbt.tile_mx4_matmul(few, m, out_dtype=torch.float32)[:, -3:], want) or worst(
        mbt.tile_mx4_matmul(few, m, out_dtype=torch.float32)[:, -3:], want.double(), 1e-3 * want.double().abs().amax()) <= 1
    y = mbt.tile_mx4_matmul(m, many, out_dtype=torch.float32)          # by pairs; results past 2^32 bytes are rows here
    size = mbt.tile_mx4_matmul(last, many, out_dtype=torch.float32)
    assert worst(y[-3:], size.double(), 1e-4 * size.double().abs().amax()) <= 1
    del m, y
    wide = mbt.tile_mx4_matmul(operand(70001, 64, 16, 53)[0], operand(65539, 64, 16, 54)[0])   # 9 GB of results
    a, b = operand(70001, 64, 16, 53)[1], operand(65539, 64, 16, 54)[1]
    for rows in (slice(0, 3), slice(69990, 70001)):
        ref = a[rows] @ b.t()
        assert worst(wide[rows], ref, 2.0 ** -7 * ref.abs() + 1e-3 * ref.abs().amax()) <= 1
    del wide, a, b
    torch.cuda.empty_cache()


def test_products_on_streams_side_by_side():
    """Products of every variant on three streams at once, back to back: clusters whose CTAs share SMs with others'."""
    shapes = [(1, 512, 4096), (17, 1024, 2048), (64, 640, 8192), (128, 512, 1024), (200, 256, 256), (100, 9000, 256),
              (2500, 2600, 512), (3, 128, 256), (33, 300, 16384)]
    cases = []
    for k, (M, N, K) in enumerate(shapes):
        block = 16 if k % 2 else 32
        a, b = operand(M, K, block, 60 + 2 * k)[0], operand(N, K, block, 61 + 2 * k)[0]
        cases.append((a, b, mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for turn in range(40):
        for s, stream in enumerate(streams):
            a, b, want = cases[(turn * (s + 1) + 2 * s) % len(cases)]
            results.append((mbt.tile_mx4_matmul(a, b, out_dtype=torch.float32, stream=stream), want))
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for got, want in results)
    assert mbt.tile_status()[0] == 0

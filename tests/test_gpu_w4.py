"""tile_w4_matvec against the formula in 64 bits."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import E4M3, OUT_U, TINY, TYPES, U, gen, pitched, randn, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def weights(N, K, group, seed, sdt=torch.bfloat16, zeros=False):
    g = gen(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    cells = (N, -(-K // group))
    s = (0.01 * (0.1 + torch.rand(cells, generator=g, device="cuda"))).to(sdt)
    z = torch.randint(0, 16, cells, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s, z


def check(x, q, s, z, group, xs, out):
    """Rounding of the output, and of fp32 sums of x (q - z) taken as x q - z x."""
    T, K = x.shape
    N = q.shape[0]
    col = torch.arange(K, device="cuda")
    w = torch.stack((q & 15, q >> 4), 2).view(N, K).double()
    zz = 8.0 if z is None else z.double()[:, col // group]
    ss = s.double()[:, col // group]
    xv = x.double()
    if xs is not None:
        xv = xv * xs.double()[:, col // (128 if xs.shape[1] > 1 else max(K, 1))]
    want = xv @ ((w - zz) * ss).t()
    bound = 64 * U * (xv.abs() @ ((w + zz) * ss).t()) + OUT_U[out.dtype] * want.abs() + TINY[out.dtype]
    assert out.shape == (T, N)
    assert worst(out, want, bound) <= 1


SHAPES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (8, 128, 128), (1, 4096, 4096), (3, 1000, 2048),
          (5, 129, 8192), (7, 4095, 1056), (8, 640, 16384), (9, 300, 512), (16, 256, 4096), (33, 50, 1024),
          (1, 100, 28672), (8, 33, 28672), (4, 20000, 256), (1, 48, 100032)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_bf16(T, N, K, group, zeros):
    x = randn((T, K), torch.bfloat16, 1)
    q, s, z = weights(N, K, group, 2, zeros=zeros)
    check(x, q, s, z, group, None, mbt.tile_w4_matvec(x, q, s, z, group=group))


@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("sdt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("odt", ["f16", "bf16", "f32"])
def test_types(xdt, sdt, odt):
    x = randn((3, 1024), TYPES[xdt], 3)
    q, s, z = weights(500, 1024, 64, 4, TYPES[sdt], True)
    out = mbt.tile_w4_matvec(x, q, s, z, group=64, out_dtype=TYPES[odt])
    assert out.dtype == TYPES[odt]
    check(x, q, s, z, 64, None, out)


@pytest.mark.parametrize("T,N,K", [(1, 1000, 4096), (5, 257, 1056), (8, 64, 8192), (2, 96, 64)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("quant", [0, 128])
def test_norm_output(T, N, K, group, quant):
    """The 8-bit output of the norm as it comes."""
    n = mbt.tile_rmsnorm(randn((T, K), torch.bfloat16, 5, 4.0), None, None, quant=quant)
    q, s, z = weights(N, K, group, 6)
    check(n.out, q, s, z, group, n.scales, mbt.tile_w4_matvec(n.out, q, s, z, group=group, x_scales=n.scales))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_range_of_activations(dtype):
    """Rows far apart in magnitude, a row of zeros, and values far apart within a row."""
    dt = TYPES[dtype]
    x = randn((6, 2048), torch.float32, 7)
    top = 2000.0 if dtype == "f16" else 1e30
    x *= torch.tensor([1.0, 0.0, top, 1.0, 1e-4 if dtype == "f16" else 1e-30, 1.0], device="cuda")[:, None]
    x[3, ::7] *= 1000.0
    x[5] = 0
    x[5, 77] = 1.0
    x = x.to(dt)
    q, s, z = weights(130, 2048, 128, 8, zeros=True)
    out = mbt.tile_w4_matvec(x, q, s, z, group=128, out_dtype=torch.float32)
    check(x, q, s, z, 128, None, out)
    assert bool((out[1] == 0).all())


def test_non_finite_rows_stay_apart():
    x = randn((8, 1024), torch.bfloat16, 9)
    q, s, z = weights(200, 1024, 128, 10)
    want = mbt.tile_w4_matvec(x, q, s, z)
    x[2, 100] = float("nan")
    x[5, 1023] = float("inf")
    got = mbt.tile_w4_matvec(x, q, s, z)
    fine = [0, 1, 3, 4, 6, 7]
    assert torch.equal(got[fine], want[fine])
    assert not bool(got[2].isfinite().any()) and not bool(got[5].isfinite().any())


@pytest.mark.parametrize("pad", [32, 1, 24])
def test_pitches(pad):
    x = pitched(randn((5, 2048), torch.bfloat16, 11), pad, pad % 8)
    q, s, z = weights(77, 2048, 128, 12)
    wide = torch.zeros(77, 1024 + 48, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + 1024] = q
    out = torch.full((5, 77 + pad), 7.0, dtype=torch.float32, device="cuda")
    mbt.tile_w4_matvec(x, wide[:, 16:16 + 1024], s, z, out=out[:, :77])
    check(x, q, s, z, 128, None, out[:, :77])
    assert bool((out[:, 77:] == 7).all())


def test_empty_and_streams():
    q, s, z = weights(64, 128, 128, 13)
    assert mbt.tile_w4_matvec(torch.empty(0, 128, dtype=torch.float16, device="cuda"), q, s).shape == (0, 64)
    none = mbt.tile_w4_matvec(torch.empty(3, 0, dtype=torch.float16, device="cuda"),
                              torch.empty(5, 0, dtype=torch.uint8, device="cuda"),
                              torch.empty(5, 0, dtype=torch.float16, device="cuda"))
    assert none.shape == (3, 5) and bool((none == 0).all())
    x = randn((8, 4096), torch.float16, 14)
    q, s, z = weights(4096, 4096, 128, 15)
    want = mbt.tile_w4_matvec(x, q, s, z)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = mbt.tile_w4_matvec(x, q, s, z, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):   # the library's workspace for st is there
        mbt.tile_w4_matvec(x, q, s, z, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and mbt.tile_status()[0] == 0


def test_weights_past_four_gib():
    N, K = 70016, 131072
    q = torch.randint(0, 256, (1, K // 2), generator=gen(16), device="cuda", dtype=torch.uint8).repeat(N, 1)
    q[-16:] = torch.randint(0, 256, (16, K // 2), generator=gen(17), device="cuda", dtype=torch.uint8)
    s = torch.full((N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    x = randn((2, K), torch.bfloat16, 18)
    out = mbt.tile_w4_matvec(x, q, s)
    check(x, q[-18:], s[-18:], None, 128, None, out[:, -18:])
    del q, s
    torch.cuda.empty_cache()


def test_refusals():
    x = randn((2, 256), torch.bfloat16, 19)
    q, s, z = weights(32, 256, 128, 20, zeros=True)
    xs = torch.ones(2, 1, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[0]), dict(x=x[:, :128]), dict(q=q.int()),
                dict(scales=s[:, :1]), dict(scales=s.double()), dict(zeros=z.int()), dict(zeros=z[:3]),
                dict(group=48), dict(x_scales=xs), dict(x=x.to(E4M3)), dict(x=x.to(E4M3), x_scales=xs.half()),
                dict(out=torch.empty(2, 31, device="cuda")), dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            mbt.tile_w4_matvec(**({"x": x, "q": q, "scales": s, "zeros": z} | bad))
    odd = torch.zeros(32, 129, dtype=torch.uint8, device="cuda")[:, :128]
    for args in ((x, odd, s), (x, q.view(-1)[8:8 + 31 * 128].view(31, 128), s[:31])):
        with pytest.raises(mbt.MbtError) as e:
            mbt.tile_w4_matvec(*args)
        assert e.value.code == -2
    with pytest.raises(mbt.MbtError) as e:
        mbt.tile_w4_matvec(x[:, :48], q[:, :24].contiguous(), s[:, :1].contiguous())
    assert e.value.code == -3


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("K", [32, 992, 1024, 1056, 2048, 2080, 4096, 5120, 8224])
@pytest.mark.parametrize("xdt", ["f16", "bf16", "e4m3"])
def test_few_rows(T, K, xdt):
    """One to four rows: K around the columns that a warp takes, N not a multiple of its rows."""
    group, N = (32, 64, 128)[K // 32 % 3], 1 + K % 7 + 16 * T
    q, s, z = weights(N, K, group, 20, torch.float32 if K == 1056 else torch.float16, zeros=K % 64 == 0)
    if xdt == "e4m3":
        n = mbt.tile_rmsnorm(randn((T, K), torch.bfloat16, 21, 4.0), None, None, quant=128 if T % 2 else 0)
        x, xs = n.out, n.scales
    else:
        x, xs = randn((T, K), TYPES[xdt], 21), None
    out = mbt.tile_w4_matvec(x, q, s, z, group=group, x_scales=xs, out_dtype=torch.float32)
    check(x, q, s, z, group, xs, out)
    assert torch.equal(out, mbt.tile_w4_matvec(x, q, s, z, group=group, x_scales=xs, out_dtype=torch.float32))


@pytest.mark.parametrize("T", [1, 4])
def test_few_rows_non_finite(T):
    """What lies past K in x and in the scales stays out; rows of x stay apart."""
    x = pitched(randn((T, 1056), torch.bfloat16, 22), 32, 0)
    q, s, z = weights(37, 1056, 128, 23)
    want = mbt.tile_w4_matvec(x, q, s, z)
    check(x, q, s, z, 128, None, want)
    s[0, 0] = float("inf")   # (the first scale of all, of row 0 only)
    got = mbt.tile_w4_matvec(x, q, s, z)
    assert torch.equal(got[:, 1:], want[:, 1:]) and not bool(got[:, 0].isfinite().any())
    x[T - 1, 1055] = float("nan")
    got = mbt.tile_w4_matvec(x, q, s, z)
    assert torch.equal(got[:T - 1, 1:], want[:T - 1, 1:]) and not bool(got[T - 1].isfinite().any())


def test_few_rows_in_a_capture():
    """No workspace: the first call on a stream may be captured."""
    x = randn((2, 2048), torch.float16, 24)
    q, s, z = weights(500, 2048, 64, 25)
    want = mbt.tile_w4_matvec(x, q, s, z, group=64)
    out, st = torch.zeros_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        mbt.tile_w4_matvec(x, q, s, z, group=64, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 4, 8])
def test_zero_points_are_four_bits(T):
    """Only the low four bits of a zero point count, in every kernel."""
    x = randn((T, 1056), torch.bfloat16, 30)
    q, s, z = weights(70, 1056, 32, 31, zeros=True)
    assert torch.equal(mbt.tile_w4_matvec(x, q, s, z | 0x50, group=32), mbt.tile_w4_matvec(x, q, s, z, group=32))


def test_many_rows_take_little_workspace():
    """Rows of x past one launch's, and a workspace that does not grow with them."""
    x = randn((70000, 64), torch.bfloat16, 32)
    q, s, z = weights(40, 64, 32, 33, zeros=True)
    check(x, q, s, z, 32, None, mbt.tile_w4_matvec(x, q, s, z, group=32))
    T, N, K = 2051, 4096, 16384
    n = mbt.tile_rmsnorm(randn((T, K), torch.bfloat16, 34, 2.0), None, quant=128)
    q, s, z = weights(N, K, 128, 35)
    out = torch.zeros(T, N + 8, dtype=torch.bfloat16, device="cuda")[:, :N]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    mbt.tile_w4_matvec(n.out, q, s, group=128, x_scales=n.scales, out=out, stream=st)
    st.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 300 << 20
    check(n.out, q, s, None, 128, n.scales, out)
    mbt.tile_workspace_release(st)

"""tile_rmsnorm and tile_rmsnorm_backward against the formulas in 64 bits."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import (E4M3, OUT_U, TINY, TYPES, U, chain, e4m3_half_spacing, norm64, pitched, randn,
                           worst)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (1, 8192), (5, 128), (1000, 64), (7, 1000), (33, 1024), (129, 4096), (3, 4097),
          (300, 2056), (2, 16384), (5, 16392), (3, 24577), (2, 65536), (1, 131080), (2, 300001),
          (700, 8191), (257, 16), (4099, 40)]


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def check_forward(x, w, r, got, eps, offset, quant):
    M, N = x.shape
    h, rstd, y = norm64(x, w, r, eps, offset)
    tol = (chain(N) / 2 + 8) * U      # of rstd; h has one rounding, y three more
    assert worst(got.rstd, rstd, tol * rstd) <= 1
    if r is not None:
        assert got.residual.dtype == x.dtype
        assert worst(got.residual, h, (OUT_U[x.dtype] + U) * h.abs() + TINY[x.dtype]) <= 1
    else:
        assert got.residual is None
    if quant is None:
        assert got.out.dtype == x.dtype
        assert worst(got.out, y, (OUT_U[x.dtype] + tol) * y.abs() + TINY[x.dtype]) <= 1
        return
    size = quant or N
    groups = -(-N // size)
    pad = torch.nn.functional.pad(y, (0, groups * size - N)).view(M, groups, size)
    scales = (pad.abs().amax(2) / 448).clamp_min(2.0 ** -126)
    assert worst(got.scales, scales, (tol + 4 * U) * scales) <= 1
    t = y / scales.repeat_interleave(size, 1)[:, :N]
    bound = e4m3_half_spacing(t * (1 + 2 * tol + 16 * U)) + (2 * tol + 16 * U) * t.abs()
    assert worst(got.out.float(), t, bound) <= 1


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(M, N, dtype, residual):
    dt = TYPES[dtype]
    x = randn((M, N), dt, 1)
    r = randn((M, N), dt, 2, 3.0) if residual else None
    w = randn(N, dt, 3)
    check_forward(x, w, r, mbt.tile_rmsnorm(x, w, r, eps=1e-5), 1e-5, 0.0, None)


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("quant", [0, 32, 64, 128])
def test_forward_e4m3(M, N, dtype, quant):
    dt = TYPES[dtype]
    x, w = randn((M, N), dt, 4), randn(N, dt, 5)
    r = randn((M, N), dt, 6) if M % 2 else None
    check_forward(x, w, r, mbt.tile_rmsnorm(x, w, r, eps=1e-6, quant=quant), 1e-6, 0.0, quant)


@pytest.mark.parametrize("wdt", ["f16", "bf16", "f32", None])
@pytest.mark.parametrize("N", [100, 2048])
def test_weight_types_and_offset(wdt, N):
    x = randn((9, N), torch.bfloat16, 7)
    w = None if wdt is None else randn(N, TYPES[wdt], 8, 0.1)
    got = mbt.tile_rmsnorm(x, w, None, eps=1e-6, weight_offset=1.0)
    check_forward(x, w, None, got, 1e-6, 1.0, None)
    h, rstd, _ = norm64(x, w, None, 1e-6, 1.0)
    dy = randn((9, N), torch.bfloat16, 9)
    dx, dw = mbt.tile_rmsnorm_backward(dy, x, rstd.float(), w, weight_offset=1.0)
    check_backward(dy, x, rstd.float(), w, None, dx, dw, 1.0)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (16, 8)])
@pytest.mark.parametrize("N", [512, 1001])
@pytest.mark.parametrize("quant", [None, 0, 64])
def test_pitches_and_offsets(pad, offset, N, quant):
    dt = torch.float16
    x = pitched(randn((37, N), dt, 10), pad, offset)
    r = pitched(randn((37, N), dt, 11), 2 * pad, offset)
    w = randn(N + 8, dt, 12)[offset:offset + N].clone()
    wide = torch.empty(37, N + 24, dtype=dt if quant is None else E4M3, device="cuda")
    wide.view(torch.uint8).fill_(0x55)
    out = wide[:, 8:8 + N]
    ro = torch.zeros(37, N + 8, dtype=dt, device="cuda")[:, :N]
    got = mbt.tile_rmsnorm(x, w, r, eps=1e-6, quant=quant, out=out, residual_out=ro)
    check_forward(x, w, r, got, 1e-6, 0.0, quant)
    raw = wide.view(torch.uint8).view(37, -1)
    es = out.element_size()
    assert bool((raw[:, :8 * es] == 0x55).all()) and bool((raw[:, (8 + N) * es:] == 0x55).all())


# enough rows for the persistent kernels, whole chunks and rows that begin inside one
LARGE = [(700, 16384), (2600, 4096), (1300, 16383), (2100, 5001), (40000, 256), (9001, 1032), (620, 20480)]


@pytest.mark.parametrize("M,N", LARGE)
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", None), ("f32", "f16")])
@pytest.mark.parametrize("residual", [False, True])
def test_many_rows(M, N, dtype, wdt, residual):
    dt = TYPES[dtype]
    x = randn((M, N), dt, 60)
    r = randn((M, N), dt, 61, 3.0) if residual else None
    w = None if wdt is None else randn(N, TYPES[wdt], 62)
    off = 0.5 if wdt == "f16" else 0.0
    got = mbt.tile_rmsnorm(x, w, r, eps=1e-5, weight_offset=off)
    check_forward(x, w, r, got, 1e-5, off, None)
    h = x if r is None else got.residual
    dy = randn((M, N), dt, 63)
    dx, dw = mbt.tile_rmsnorm_backward(dy, h, got.rstd, w, dresidual=r, weight_offset=off)
    if wdt is None:
        dw = torch.empty(N, device="cuda")
        dx, dw = mbt.tile_rmsnorm_backward(dy, h, got.rstd, w, dresidual=r, dweight=dw)
    check_backward(dy, h, got.rstd, w, r, dx, dw, off)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", [(30000, 100), (50001, 24), (20011, 64), (9000, 1000), (40, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_many_short_rows_backward(M, N, dtype, dres):
    """Several rows to a warp, whole and partial chunks; fewer rows than the device takes at once."""
    dt = TYPES[dtype]
    dy, h, w = randn((M, N), dt, 65), randn((M, N), dt, 66, 2.0), randn(N, dt, 67)
    r = randn((M, N), dt, 68) if dres else None
    rstd = 1 / torch.sqrt(h.float().square().mean(1) + 1e-5)
    dx, dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w, dresidual=r)
    check_backward(dy, h, rstd, w, r, dx, dw, 0.0)
    again = mbt.tile_rmsnorm_backward(dy, h, rstd, w, dresidual=r)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", LARGE)
@pytest.mark.parametrize("quant", [0, 32, 64, 128])
def test_many_rows_e4m3(M, N, quant):
    x, w, r = randn((M, N), torch.bfloat16, 64), randn(N, torch.bfloat16, 65), randn((M, N), torch.bfloat16, 66)
    check_forward(x, w, r, mbt.tile_rmsnorm(x, w, r, eps=1e-6, quant=quant), 1e-6, 0.0, quant)


@pytest.mark.parametrize("pad", [8, 3])
def test_many_rows_with_pitches(pad):
    M, N, dt = 2600, 4001, torch.bfloat16
    x, r, dy = (pitched(randn((M, N), dt, 67 + k), pad) for k in range(3))
    w = randn(N, dt, 70)
    wide = [torch.zeros(M, N + pad, dtype=dt, device="cuda") for _ in range(3)]
    got = mbt.tile_rmsnorm(x, w, r, out=wide[0][:, :N], residual_out=wide[1][:, :N], eps=1e-6)
    check_forward(x, w, r, got, 1e-6, 0.0, None)
    dx, dw = mbt.tile_rmsnorm_backward(dy, x, got.rstd, w, dresidual=r, dx=wide[2][:, :N])
    check_backward(dy, x, got.rstd, w, r, dx, dw)
    assert all(bool((t[:, N:] == 0).all()) for t in wide)


def test_in_place():
    for rows, N in ((65, 1024), (65, 1001), (2600, 4001)):
        x, r, w = randn((rows, N), torch.bfloat16, 13), randn((rows, N), torch.bfloat16, 14), randn(N, torch.bfloat16, 15)
        want = mbt.tile_rmsnorm(x, w, r)
        x2, r2 = x.clone(), r.clone()
        got = mbt.tile_rmsnorm(x2, w, r2, out=x2, residual_out=r2)
        assert torch.equal(got.out, want.out) and torch.equal(r2, want.residual)
        dy, dr = randn((rows, N), torch.bfloat16, 16), randn((rows, N), torch.bfloat16, 17)
        dx, dw = mbt.tile_rmsnorm_backward(dy, r2, got.rstd, w, dresidual=dr)
        for target in ("dy", "dres"):
            a, b = dy.clone(), dr.clone()
            dx2, dw2 = mbt.tile_rmsnorm_backward(a, r2, got.rstd, w, dresidual=b, dx=a if target == "dy" else b)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("N", [256, 1000, 9001])
def test_special_rows(N):
    """Rows of zeros, of one value, with a NaN, with an infinity: each row by itself."""
    x = randn((6, N), torch.float32, 18)
    x[1] = 0
    x[2] = 0
    x[2, N // 2] = 5.0
    x[3, N - 1] = float("nan")
    x[4, 0] = float("inf")
    got = mbt.tile_rmsnorm(x, None, None, eps=1e-6)
    assert bool((got.out[1] == 0).all()) and bool(got.out[3].isnan().all())
    assert got.out[4, 0].isnan() and bool((got.out[4, 1:] == 0).all()) and got.rstd[4] == 0
    fine = [0, 1, 2, 5]
    check_forward(x[fine], None, None,
                  mbt.RmsNorm(got.out[fine], None, None, got.rstd[fine]), 1e-6, 0.0, None)
    for quant in (0, 128):
        q = mbt.tile_rmsnorm(x, None, None, eps=1e-6, quant=quant)
        assert bool((q.out[1].float() == 0).all()) and bool((q.scales[1] == 2.0 ** -126).all())
        assert bool(q.out[3].float().isnan().all()) and bool(q.scales[3].isnan().all())
        assert q.scales[4, 0].isnan()
        assert bool(q.out[fine].float().isfinite().all())


def test_empty():
    x = torch.empty(0, 64, device="cuda")
    got = mbt.tile_rmsnorm(x, torch.ones(64, device="cuda"), None)
    assert got.out.shape == (0, 64) and got.rstd.shape == (0,)
    dw = torch.ones(64, device="cuda")
    mbt.tile_rmsnorm_backward(x, x, got.rstd, dw.clone(), dweight=dw)
    assert bool((dw == 0).all())
    got = mbt.tile_rmsnorm(torch.empty(3, 0, device="cuda"), None, None, eps=0.25)
    assert bool((got.rstd == 2).all())


def check_backward(dy, h, rstd, w, dres, dx, dw, offset=0.0):
    M, N = h.shape
    g = dy.double() * (1 if w is None else w.double() + offset)
    rs = rstd.double()[:, None]
    xh = h.double() * rs
    c = (g * xh).mean(1, keepdim=True)
    want = rs * (g - xh * c) + (dres.double() if dres is not None else 0)
    mean_abs = (g * xh).abs().mean(1, keepdim=True)
    bound = 8 * U * ((rs * g).abs() + (rs * xh * c).abs()) + (chain(N) + 8) * U * (rs * xh).abs() * mean_abs
    bound += (2 * U + OUT_U[h.dtype]) * want.abs() + TINY[h.dtype]
    if dres is not None:
        bound += U * dres.double().abs()
    assert worst(dx, want, bound) <= 1
    if dw is not None:
        # roundings of a column's M terms are independent: their sum grows with sqrt(M)
        terms = dy.double() * xh
        assert dw.dtype == torch.float32
        assert worst(dw, terms.sum(0), (40 + 4 * M ** 0.5) * U * terms.abs().sum(0) + 1e-30) <= 1


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(M, N, dtype, dres):
    dt = TYPES[dtype]
    h, dy, w = randn((M, N), dt, 20), randn((M, N), dt, 21), randn(N, dt, 22)
    rstd = mbt.tile_rmsnorm(h, w, None).rstd
    d = randn((M, N), dt, 23) if dres else None
    dx, dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w, dresidual=d)
    check_backward(dy, h, rstd, w, d, dx, dw)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("N", [512, 1001])
def test_backward_pitches(pad, offset, N):
    dt = torch.bfloat16
    h, dy = pitched(randn((70, N), dt, 24), pad, offset), pitched(randn((70, N), dt, 25), 0, 8)
    w, d = randn(N, torch.float32, 26), pitched(randn((70, N), dt, 27), pad)
    rstd = mbt.tile_rmsnorm(h, w, None).rstd
    wide = torch.zeros(70, N + 24, dtype=dt, device="cuda")
    dx, dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w, dresidual=d, dx=wide[:, 8:8 + N])
    check_backward(dy, h, rstd, w, d, dx, dw)
    assert bool((wide[:, :8] == 0).all()) and bool((wide[:, 8 + N:] == 0).all())


def test_gradient_against_autograd_and_differences():
    M, N = 5, 768
    x, r, w = randn((M, N), torch.float32, 30), randn((M, N), torch.float32, 31), randn(N, torch.float32, 32)
    dy, dh = randn((M, N), torch.float32, 33), randn((M, N), torch.float32, 34)
    fwd = mbt.tile_rmsnorm(x, w, r, eps=1e-5)
    dx, dw = mbt.tile_rmsnorm_backward(dy, fwd.residual, fwd.rstd, w, dresidual=dh)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    h = x64 + r.double()
    y = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * w64
    ((y * dy.double()).sum() + (h * dh.double()).sum()).backward()
    assert worst(dx, x64.grad, 1e-5 * x64.grad.abs().mean() + 1e-5 * x64.grad.abs()) <= 1
    assert worst(dw, w64.grad, 1e-5 * w64.grad.abs().mean() + 1e-5 * w64.grad.abs()) <= 1
    # central differences of the forward call along a random direction: step 2^-7,
    # so rounding gives about u / 2^-7 and the third derivative about 2^-14
    def loss(xv, wv):
        f = mbt.tile_rmsnorm(xv, wv, r, eps=1e-5)
        return ((f.out.double() * dy.double()).sum() + (f.residual.double() * dh.double()).sum()).item()

    e = 2.0 ** -7
    vx, vw = randn((M, N), torch.float32, 35), randn(N, torch.float32, 36)
    for got, plus, minus in ((dx.double() * vx.double(), (x + e * vx, w), (x - e * vx, w)),
                             (dw.double() * vw.double(), (x, w + e * vw), (x, w - e * vw))):
        diff = (loss(*plus) - loss(*minus)) / (2 * e)
        assert abs(got.sum().item() - diff) <= 2e-3 * got.square().sum().sqrt().item() + 1e-3 * abs(diff)


def test_equal_calls_give_equal_bits_and_graph_capture():
    x, w, dy = randn((513, 2048), torch.bfloat16, 40), randn(2048, torch.bfloat16, 41), randn((513, 2048), torch.bfloat16, 42)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fwd = mbt.tile_rmsnorm(x, w, None, stream=s)
    dx, dw = mbt.tile_rmsnorm_backward(dy, x, fwd.rstd, w, stream=s)
    s.synchronize()
    out2, rstd2, dx2, dw2 = (torch.zeros_like(t) for t in (fwd.out, fwd.rstd, dx, dw))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mbt.tile_rmsnorm(x, w, None, out=out2, rstd=rstd2)
        mbt.tile_rmsnorm_backward(dy, x, rstd2, w, dx=dx2, dweight=dw2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in ((fwd.out, out2), (fwd.rstd, rstd2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)
    assert mbt.tile_status()[0] == 0


def test_past_four_gib():
    """Rows whose offsets pass 32 bits, in elements and in bytes."""
    M, N = 70000, 65536 - 8
    x = torch.ones(1, 1, dtype=torch.float16, device="cuda").expand(M, N).contiguous()
    x[-1] = randn((1, N), torch.float16, 43)[0]
    out = torch.empty_like(x)
    got = mbt.tile_rmsnorm(x, None, None, out=out, eps=1e-6)
    check_forward(x[-3:], None, None, mbt.RmsNorm(out[-3:], None, None, got.rstd[-3:]), 1e-6, 0.0, None)
    del x, out, got
    torch.cuda.empty_cache()


def test_refusals():
    x, w = randn((4, 64), torch.float16, 50), randn(64, torch.float16, 51)
    ok = mbt.tile_rmsnorm(x, w)
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(weight=w[:-1]),
                dict(weight=w.double()), dict(residual=x[:2]), dict(residual=x.float()), dict(quant=16),
                dict(residual_out=x), dict(scales=ok.rstd), dict(out=x.float()), dict(rstd=ok.rstd[:2]),
                dict(quant=0, out=x), dict(quant=0, scales=ok.rstd)):
        with pytest.raises(ValueError):
            mbt.tile_rmsnorm(**({"x": x, "weight": w} | bad))
    with pytest.raises(mbt.MbtError):
        mbt.tile_rmsnorm(x, w, eps=-1.0)
    for bad in (dict(dy=x[:2]), dict(dy=x.float()), dict(rstd=ok.rstd.half()), dict(weight=w[1:]),
                dict(dresidual=x.t()), dict(dx=x.float()), dict(dweight=w)):
        with pytest.raises(ValueError):
            mbt.tile_rmsnorm_backward(**({"dy": x, "h": x, "rstd": ok.rstd, "weight": w} | bad))


@pytest.mark.parametrize("M,N", [(512, 8192), (40, 300001), (700, 16384), (3000, 4104)])
@pytest.mark.parametrize("quant", [0, 32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_e4m3_codes_are_quotients(M, N, quant, dtype):
    """Every code is y / scale of the scale that comes with it, rounded to nearest even, in each of the kernels."""
    dt = TYPES[dtype]
    x, r, w = randn((M, N), dt, 71), randn((M, N), dt, 72, 2.0), randn(N, dt, 73)
    got = mbt.tile_rmsnorm(x, w, r, quant=quant)
    y = (x.float() + r.float()) * got.rstd[:, None] * w.float()
    scales = got.scales.repeat_interleave(quant or N, 1)[:, :N]
    want = (y / scales).clamp(-448, 448).to(E4M3)
    assert torch.equal(got.out.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("rms,eps", [(1e15, 1e-6), (1e17, 1e-6), (1e-15, 0.0), (3e-18, 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,offset", [(64, 4096, 0), (64, 4096, 1), (900, 1000, 0), (7, 30000, 0)])
def test_backward_at_any_magnitude(rms, eps, dtype, M, N, offset):
    """Large and small rows, with dy along h so that the projection counts (an offset of 1: the element-wise kernels)."""
    dt = TYPES[dtype]
    n = randn((M, N), torch.float32, 74)
    if N > 4096:
        n = n.clamp(-2, 2)   # (the sum of 30000 squares of 1e17 stays in fp32's range)
    h, w = pitched((n * rms).to(dt), 0, offset), 1 + randn(N, torch.float32, 75, 0.2)
    dy = (0.7 * n + randn((M, N), torch.float32, 76, 0.5)).to(dt)
    rstd = mbt.tile_rmsnorm(h, w, None, eps=eps).rstd
    dx, dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w)
    assert (dy.double() * w.double() * h.double() * rstd.double()[:, None]).mean().item() > 0.4
    check_backward(dy, h, rstd, w, None, dx, dw)


@pytest.mark.parametrize("N", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 4])
def test_narrow_matrices_backward(N, dtype, pad):
    """Rows shorter than 16 bytes, several of which end in the matrix's last chunk."""
    dt = TYPES[dtype]
    for M in (1, 2, 3, 4, 5, 6, 7, 8, 9, 500, 4001):
        dy, h, d = (pitched(randn((M, N), dt, 97 + k), pad * (k + 1)) for k in range(3))
        w = randn(N, dt, 77)
        rstd = 1 / torch.sqrt(h.float().square().mean(1) + 1e-2)
        store = torch.full((M * (N + pad) + 64,), 7.0, dtype=dt, device="cuda")
        dx = store[:M * (N + pad)].view(M, N + pad)[:, :N]
        got, dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w, dresidual=d, dx=dx)
        check_backward(dy, h, rstd, w, d, got, dw)
        dx.fill_(7.0)
        assert bool((store == 7).all())
        a = dy.contiguous().clone()
        want, wdw = mbt.tile_rmsnorm_backward(a.clone(), h.contiguous(), rstd, w)
        mine, mdw = mbt.tile_rmsnorm_backward(a, h.contiguous(), rstd, w, dx=a)
        assert torch.equal(mine, want) and torch.equal(mdw, wdw)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N,dtype", [(16000, 64, "f32"), (16000, 64, "bf16"), (4096, 30000, "f32")])
def test_dweight_error_of_many_rows(M, N, dtype):
    """The sum over the rows is as exact as a balanced one.

    One rounding is off by 0.43 u of the rounded value on the average (uniform within half an ulp, mantissas spread
    logarithmically); of independent terms, each level of a balanced order adds one such error of the result, a series
    of k additions k / 2.  Up to 24 of them in all (a term's own, the rows of a thread, then eights, fours and pairs):
    2.1 u, and a tenth for the spread over the columns.  (64 row slots in series alone would be 32.)"""
    dt, off, norm = TYPES[dtype], 0.0, 0.0
    for seed in range(4 if N < 1000 else 1):
        h, dy, w = randn((M, N), dt, 80 + 3 * seed), randn((M, N), dt, 81 + 3 * seed), randn(N, dt, 82)
        rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
        dw = mbt.tile_rmsnorm_backward(dy, h, rstd, w)[1]
        want = (dy.double() * h.double() * rstd.double()[:, None]).sum(0)
        off += (dw.double() - want).square().sum().item()
        norm += want.square().sum().item()
    assert (off / norm) ** 0.5 <= 2.3 * U


def test_given_results_raise_their_version():
    """Autograd notices that a tensor it saved was overwritten."""
    x, w = randn((4, 64), torch.float32, 95), randn(64, torch.float32, 96)
    out, ro, rstd, dx, dw = torch.empty_like(x), x.clone(), torch.empty(4, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    before = [t._version for t in (out, ro, rstd, dx, dw)]
    mbt.tile_rmsnorm(x, w, x, out=out, residual_out=ro, rstd=rstd)
    mbt.tile_rmsnorm_backward(x, ro, rstd, w, dx=dx, dweight=dw)
    assert [t._version for t in (out, ro, rstd, dx, dw)] == [b + 1 for b in before]
    p = torch.ones(64, device="cuda", requires_grad=True)
    loss = (p * p).sum()
    state = mbt.AdamwTensors([p.detach()], [torch.zeros(64, device="cuda")], [torch.zeros(64, device="cuda")])
    mbt.tile_adamw(state, [torch.ones(64, device="cuda")], step=1, lr=0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():   # (no versions there)
        mbt.tile_rmsnorm(x.clone(), w, out=torch.empty_like(x))


@pytest.mark.parametrize("M,N,quant", [(2600, 4096, 32), (2600, 4096, 128), (2500, 4104, 64), (2500, 4104, 128),
                                       (1300, 8191, 0), (2100, 5001, 0), (620, 20480, 64), (650, 16392, 128)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual,wdt", [(False, "same"), (True, "f32"), (True, None), (False, "other")])
def test_many_rows_e4m3_types(M, N, quant, dtype, residual, wdt):
    """The persistent kernel's 8-bit output for every type of rows and weights, lengths that end inside a group."""
    dt = TYPES[dtype]
    x = randn((M, N), dt, 85)
    r = randn((M, N), dt, 86, 2.0) if residual else None
    other = torch.float16 if dtype == "bf16" else torch.bfloat16
    w = None if wdt is None else randn(N, {"same": dt, "f32": torch.float32, "other": other}[wdt], 87)
    check_forward(x, w, r, mbt.tile_rmsnorm(x, w, r, eps=1e-6, quant=quant), 1e-6, 0.0, quant)
    assert mbt.tile_status()[0] == 0

"""tile_layernorm and tile_layernorm_backward against the formulas in 64 bits.

Forward: the mean is off by at most delta = (chain + 2) u mean|h|; a shift by delta adds delta^2
to the variance (the deviations' sum is 0), a rounding of h (with a residual) u |h| d to it."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import (E4M3, OUT_U, TINY, TYPES, U, chain, e4m3_half_spacing, pitched, randn, worst)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (1, 8192), (5, 128), (1000, 64), (7, 1000), (33, 1024), (129, 4096), (3, 4097),
          (300, 2056), (2, 16384), (5, 16392), (3, 24577), (2, 65536), (2, 300001), (700, 8191), (257, 16), (4099, 40)]
# enough rows for persistent kernels, whole chunks and rows that begin inside one
LARGE = [(700, 16384), (2600, 4096), (1300, 16383), (2100, 5001), (40000, 256), (9001, 1032), (620, 20480), (5000, 8192)]


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def check_forward(x, w, b, r, got, eps, offset, quant):
    M, N = x.shape
    h = x.double() + (r.double() if r is not None else 0)
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1 / (d.square().mean(1) + eps).sqrt()
    wide = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double() + offset
    bias = torch.zeros(N, dtype=torch.float64, device="cuda") if b is None else b.double()
    y = d * rstd[:, None] * wide + bias
    delta = (chain(N) + 2) * U * h.abs().mean(1)
    assert worst(got.mean, mean, delta + U * mean.abs()) <= 1
    tol = (chain(N) / 2 + 8) * U + 4 * U * h.square().mean(1).sqrt() * rstd + (delta * rstd) ** 2
    assert worst(got.rstd, rstd, tol * rstd) <= 1
    if r is not None:
        assert got.residual.dtype == x.dtype
        assert worst(got.residual, h, (OUT_U[x.dtype] + U) * h.abs() + TINY[x.dtype]) <= 1
    else:
        assert got.residual is None
    err = (rstd[:, None] * wide).abs() * (delta[:, None] + 2 * U * h.abs() + 2 * U * mean[:, None].abs())
    err = err + (tol[:, None] + 6 * U) * (y - bias).abs() + 2 * U * (y.abs() + bias.abs())
    if quant is None:
        assert got.out.dtype == x.dtype
        assert worst(got.out, y, err + OUT_U[x.dtype] * (y.abs() + err) + TINY[x.dtype]) <= 1
        return
    size = quant or N
    groups = -(-N // size)

    def most(t):
        return torch.nn.functional.pad(t, (0, groups * size - N)).view(M, groups, size).abs().amax(2)

    scales = (most(y) / 448).clamp_min(2.0 ** -126)
    off = most(err) / 448 + 4 * U * scales
    assert worst(got.scales, scales, off) <= 1
    s = scales.repeat_interleave(size, 1)[:, :N]
    t = y / s
    slack = err / s + t.abs() * (off / scales).repeat_interleave(size, 1)[:, :N] + 4 * U * t.abs()
    assert worst(got.out.float(), t, e4m3_half_spacing(t.abs() + slack) + slack) <= 1


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(M, N, dtype, residual):
    dt = TYPES[dtype]
    x = randn((M, N), dt, 1) + 0.5
    r = randn((M, N), dt, 2, 3.0) if residual else None
    w, b = randn(N, dt, 3), randn(N, dt, 4)
    check_forward(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-5), 1e-5, 0.0, None)


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("quant", [0, 32, 64, 128])
def test_forward_e4m3(M, N, dtype, quant):
    dt = TYPES[dtype]
    x, w, b = randn((M, N), dt, 4) - 1, randn(N, dt, 5), randn(N, dt, 7)
    r = randn((M, N), dt, 6) if M % 2 else None
    check_forward(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-6, quant=quant), 1e-6, 0.0, quant)


@pytest.mark.parametrize("wdt", ["f16", "bf16", "f32", None])
@pytest.mark.parametrize("N", [100, 2048])
@pytest.mark.parametrize("biased", [False, True])
def test_weight_types_and_offset(wdt, N, biased):
    x = randn((9, N), torch.bfloat16, 7)
    w = None if wdt is None else randn(N, TYPES[wdt], 8, 0.1)
    b = randn(N, TYPES[wdt], 9) if biased and w is not None else None
    got = mbt.tile_layernorm(x, w, b, eps=1e-6, weight_offset=1.0)
    check_forward(x, w, b, None, got, 1e-6, 1.0, None)
    dy = randn((9, N), torch.bfloat16, 9)
    dx, dw, db = mbt.tile_layernorm_backward(dy, x, got.mean, got.rstd, w, weight_offset=1.0, bias=biased)
    assert (dw is None) == (w is None) and (db is None) == (w is None or not biased)
    check_backward(dy, x, got.mean, got.rstd, w, None, dx, dw, db, 1.0)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (16, 8)])
@pytest.mark.parametrize("N", [512, 1001])
@pytest.mark.parametrize("quant", [None, 0, 64])
def test_pitches_and_offsets(pad, offset, N, quant):
    dt = torch.float16
    x = pitched(randn((37, N), dt, 10), pad, offset)
    r = pitched(randn((37, N), dt, 11), 2 * pad, offset)
    w, b = randn(N + 8, dt, 12)[offset:offset + N].clone(), randn(N + 8, dt, 13)[offset:offset + N]
    wide = torch.empty(37, N + 24, dtype=dt if quant is None else E4M3, device="cuda")
    wide.view(torch.uint8).fill_(0x55)
    out = wide[:, 8:8 + N]
    ro = torch.zeros(37, N + 8, dtype=dt, device="cuda")[:, :N]
    got = mbt.tile_layernorm(x, w, b, r, eps=1e-6, quant=quant, out=out, residual_out=ro)
    check_forward(x, w, b, r, got, 1e-6, 0.0, quant)
    raw = wide.view(torch.uint8).view(37, -1)
    es = out.element_size()
    assert bool((raw[:, :8 * es] == 0x55).all()) and bool((raw[:, (8 + N) * es:] == 0x55).all())


@pytest.mark.parametrize("M,N", LARGE)
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", None), ("f32", "f16")])
@pytest.mark.parametrize("residual", [False, True])
def test_many_rows(M, N, dtype, wdt, residual):
    dt = TYPES[dtype]
    x = randn((M, N), dt, 60) + 2
    r = randn((M, N), dt, 61, 3.0) if residual else None
    w = None if wdt is None else randn(N, TYPES[wdt], 62)
    b = None if wdt is None else randn(N, TYPES[wdt], 64)
    off = 0.5 if wdt == "f16" else 0.0
    got = mbt.tile_layernorm(x, w, b, r, eps=1e-5, weight_offset=off)
    check_forward(x, w, b, r, got, 1e-5, off, None)
    h = x if r is None else got.residual
    dy = randn((M, N), dt, 63)
    given = {} if wdt else dict(dweight=torch.empty(N, device="cuda"), dbias=torch.empty(N, device="cuda"))
    dx, dw, db = mbt.tile_layernorm_backward(dy, h, got.mean, got.rstd, w, dresidual=r, weight_offset=off, **given)
    check_backward(dy, h, got.mean, got.rstd, w, r, dx, dw, db, off)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", [(30000, 100), (50001, 24), (20011, 64), (9000, 1000), (40, 8192), (65537, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_many_short_rows_backward(M, N, dtype, dres):
    dt = TYPES[dtype]
    dy, h, w = randn((M, N), dt, 65), randn((M, N), dt, 66, 2.0), randn(N, dt, 67)
    r = randn((M, N), dt, 68) if dres else None
    stats = h.float().mean(1), 1 / torch.sqrt(h.float().var(1, correction=0) + 1e-5)
    got = mbt.tile_layernorm_backward(dy, h, *stats, w, dresidual=r)
    check_backward(dy, h, *stats, w, r, *got)
    for a, b in zip(got, mbt.tile_layernorm_backward(dy, h, *stats, w, dresidual=r)):
        assert torch.equal(a, b)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", LARGE + [(2600, 1000), (1300, 8191)])
@pytest.mark.parametrize("quant", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "bf16"), ("bf16", None)])
def test_many_rows_e4m3(M, N, quant, dtype, wdt):
    dt = TYPES[dtype]
    x, r = randn((M, N), dt, 64), randn((M, N), dt, 66) if N % 3 else None
    w, b = (None, None) if wdt is None else (randn(N, TYPES[wdt], 65), randn(N, TYPES[wdt], 67))
    check_forward(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-6, quant=quant), 1e-6, 0.0, quant)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("pad", [8, 3])
def test_many_rows_with_pitches(pad):
    M, N, dt = 2600, 4001, torch.bfloat16
    x, r, dy = (pitched(randn((M, N), dt, 67 + k), pad) for k in range(3))
    w, b = randn(N, dt, 70), randn(N, dt, 71)
    wide = [torch.zeros(M, N + pad, dtype=dt, device="cuda") for _ in range(3)]
    got = mbt.tile_layernorm(x, w, b, r, out=wide[0][:, :N], residual_out=wide[1][:, :N], eps=1e-6)
    check_forward(x, w, b, r, got, 1e-6, 0.0, None)
    dx, dw, db = mbt.tile_layernorm_backward(dy, x, got.mean, got.rstd, w, dresidual=r, dx=wide[2][:, :N])
    check_backward(dy, x, got.mean, got.rstd, w, r, dx, dw, db)
    assert all(bool((t[:, N:] == 0).all()) for t in wide)


@pytest.mark.parametrize("M,N", [(6000, 4104), (7000, 4103), (13000, 2056), (40001, 520), (40000, 511), (1900, 16379), (310, 20001),
                                 (155, 32761), (700, 16392), (310, 20008), (200, 26624), (160, 26632), (157, 32768), (154, 12000), (320, 13320),
                                 (156, 16384), (311, 12001), (155, 16381), (400, 8888), (309, 10239)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("quant", [None, 0, 32, 128])
def test_long_rows(M, N, dtype, quant):
    """Rows that stay in shared memory from pass to pass, in several stages or one; one turn and more."""
    dt = TYPES[dtype]
    w, b = randn(N, dt, 73), randn(N, dt, 74)
    for r in (None, randn((M, N), dt, 72, 3.0)):
        x = randn((M, N), dt, 71) + 1
        check_forward(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-5, quant=quant), 1e-5, 0.0, quant)
    if quant is None:
        check_forward(x, None, None, r, mbt.tile_layernorm(x, None, None, r, eps=1e-5), 1e-5, 0.0, None)
        check_forward(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-5, weight_offset=0.5), 1e-5, 0.5, None)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", [(330, 20008), (160, 32768), (311, 12001), (155, 16381), (311, 9001), (200, 10240)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_rows_in_place(M, N, dtype):
    dt = TYPES[dtype]
    x, r, w, b = randn((M, N), dt, 75), randn((M, N), dt, 76), randn(N, dt, 77), randn(N, dt, 78)
    want = mbt.tile_layernorm(x, w, b, r)
    check_forward(x, w, b, r, want, 1e-5, 0.0, None)
    x2, r2 = x.clone(), r.clone()
    got = mbt.tile_layernorm(x2, w, b, r2, out=x2, residual_out=r2)
    for a, c in zip((got.out, r2, got.mean, got.rstd), (want.out, want.residual, want.mean, want.rstd)):
        assert torch.equal(a, c)
    dy = randn((M, N), dt, 79)
    first = mbt.tile_layernorm_backward(dy, r2, got.mean, got.rstd, w, dresidual=x)
    check_backward(dy, r2, got.mean, got.rstd, w, x, *first)
    again = mbt.tile_layernorm_backward(dy, r2, got.mean, got.rstd, w, dresidual=x, dx=x)
    for a, c in zip(first, again):
        assert torch.equal(a, c)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("rows,N", [(65, 1024), (65, 1001), (2600, 4001), (700, 16384), (3, 70000)])
def test_in_place(rows, N):
    x, r = randn((rows, N), torch.bfloat16, 13), randn((rows, N), torch.bfloat16, 14)
    w, b = randn(N, torch.bfloat16, 15), randn(N, torch.bfloat16, 18)
    want = mbt.tile_layernorm(x, w, b, r)
    x2, r2 = x.clone(), r.clone()
    got = mbt.tile_layernorm(x2, w, b, r2, out=x2, residual_out=r2)
    assert torch.equal(got.out, want.out) and torch.equal(r2, want.residual)
    dy, dr = randn((rows, N), torch.bfloat16, 16), randn((rows, N), torch.bfloat16, 17)
    first = mbt.tile_layernorm_backward(dy, r2, got.mean, got.rstd, w, dresidual=dr)
    for target in ("dy", "dres"):
        p, q = dy.clone(), dr.clone()
        again = mbt.tile_layernorm_backward(p, r2, got.mean, got.rstd, w, dresidual=q, dx=p if target == "dy" else q)
        for a, b2 in zip(first, again):
            assert torch.equal(a, b2)


@pytest.mark.parametrize("N", [256, 1000, 9001])
@pytest.mark.parametrize("M", [6, 3000])
def test_special_rows(M, N):
    """Rows of one value, of zeros, with a NaN, with an infinity: each row by itself."""
    x = randn((M, N), torch.float32, 18)
    x[1] = 0
    x[2] = 3.0
    x[3, N - 1] = float("nan")
    x[4, 0] = float("inf")
    b = torch.full((N,), 0.25, device="cuda")
    got = mbt.tile_layernorm(x, torch.ones(N, device="cuda"), b, eps=1e-6)
    assert bool((got.out[1:3] == 0.25).all()) and bool((got.rstd[1:3] == torch.tensor(1e-6).rsqrt().item()).all() or
                                                       ((got.rstd[1:3] - 1000).abs() < 1e-3).all())
    assert bool(got.out[3].isnan().all()) and bool(got.out[4].isnan().all())
    fine = [0, 5]
    check_forward(x[fine], torch.ones(N, device="cuda"), b, None,
                  mbt.LayerNorm(got.out[fine], None, None, got.mean[fine], got.rstd[fine]), 1e-6, 0.0, None)
    for quant in (0, 128):
        q = mbt.tile_layernorm(x, None, None, eps=1e-6, quant=quant)
        assert bool((q.out[1:3].float() == 0).all()) and bool((q.scales[1:3] == 2.0 ** -126).all())
        assert bool(q.scales[3].isnan().all()) and bool(q.scales[4].isnan().all())
        assert bool(q.out[fine].float().isfinite().all())


@pytest.mark.parametrize("M,N", [(5, 4096), (3, 1001), (3000, 4096), (2, 60000)])
@pytest.mark.parametrize("mean", [1000.0, -3e4])
def test_means_far_from_zero(M, N, mean):
    """Rows whose mean is large against their deviation keep the variance."""
    x = randn((M, N), torch.float32, 19) + mean
    got = mbt.tile_layernorm(x, None, None, eps=0.0)
    check_forward(x, None, None, None, got, 0.0, 0.0, None)
    var = x.double().var(1, correction=0)
    assert worst(got.rstd, var.rsqrt(), 2e-4 * var.rsqrt()) <= 1


def test_empty():
    x = torch.empty(0, 64, device="cuda")
    got = mbt.tile_layernorm(x, torch.ones(64, device="cuda"))
    assert got.out.shape == (0, 64) and got.mean.shape == got.rstd.shape == (0,)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    mbt.tile_layernorm_backward(x, x, got.mean, got.rstd, dw.clone(), dweight=dw, dbias=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    got = mbt.tile_layernorm(torch.empty(3, 0, device="cuda"), eps=0.25)
    assert bool((got.rstd == 2).all()) and bool((got.mean == 0).all())


def check_backward(dy, h, mean, rstd, w, dres, dx, dw, db, offset=0.0):
    M, N = h.shape
    g = dy.double() * (1 if w is None else w.double() + offset)
    rs = rstd.double()[:, None]
    xh = (h.double() - mean.double()[:, None]) * rs
    level, along = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    want = rs * (g - level - xh * along) + (dres.double() if dres is not None else 0)
    sums = (chain(N) + 8) * U * (g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    bound = rs * (8 * U * (g.abs() + level.abs() + (xh * along).abs()) + sums)
    bound += (2 * U + OUT_U[h.dtype]) * want.abs() + OUT_U[h.dtype] * bound + TINY[h.dtype]
    if dres is not None:
        bound += U * dres.double().abs()
    assert worst(dx, want, bound) <= 1
    # roundings of a column's M terms are independent: their sum grows with sqrt(M)
    for got, terms in ((dw, dy.double() * xh), (db, dy.double())):
        if got is not None:
            assert got.dtype == torch.float32
            assert worst(got, terms.sum(0), (40 + 4 * M ** 0.5) * U * terms.abs().sum(0) + 1e-30) <= 1


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(M, N, dtype, dres):
    dt = TYPES[dtype]
    h, dy, w = randn((M, N), dt, 20) + 1, randn((M, N), dt, 21), randn(N, dt, 22)
    fwd = mbt.tile_layernorm(h, w)
    d = randn((M, N), dt, 23) if dres else None
    got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, dresidual=d)
    check_backward(dy, h, fwd.mean, fwd.rstd, w, d, *got)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("N", [512, 1001])
def test_backward_pitches(pad, offset, N):
    dt = torch.bfloat16
    h, dy = pitched(randn((70, N), dt, 24), pad, offset), pitched(randn((70, N), dt, 25), 0, 8)
    w, d = randn(N, torch.float32, 26), pitched(randn((70, N), dt, 27), pad)
    fwd = mbt.tile_layernorm(h, w)
    wide = torch.zeros(70, N + 24, dtype=dt, device="cuda")
    got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, dresidual=d, dx=wide[:, 8:8 + N])
    check_backward(dy, h, fwd.mean, fwd.rstd, w, d, *got)
    assert bool((wide[:, :8] == 0).all()) and bool((wide[:, 8 + N:] == 0).all())


def test_gradients_one_at_a_time():
    """dweight or dbias alone, and neither."""
    dy, h, w = randn((300, 512), torch.bfloat16, 28), randn((300, 512), torch.bfloat16, 29), randn(512, torch.bfloat16, 30)
    fwd = mbt.tile_layernorm(h, w)
    dx, dw, db = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w)
    a = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, bias=False)
    assert torch.equal(a[0], dx) and torch.equal(a[1], dw) and a[2] is None
    ones = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    want = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, ones)
    b = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, None, dbias=torch.empty(512, device="cuda"))
    assert b[1] is None and torch.equal(b[2], db) and worst(b[0], want[0].double(), 2 ** -7 * want[0].double().abs() + 1e-6) <= 1
    c = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd)
    assert c[1] is None and c[2] is None and torch.equal(c[0], b[0])


@pytest.mark.parametrize("M", [5, 400])
def test_gradient_against_autograd_and_differences(M):
    N = 768
    x, r, w, b = (randn(s, torch.float32, 30 + k) for k, s in enumerate(((M, N), (M, N), N, N)))
    dy, dh = randn((M, N), torch.float32, 34), randn((M, N), torch.float32, 35)
    fwd = mbt.tile_layernorm(x, w, b, r, eps=1e-5)
    dx, dw, db = mbt.tile_layernorm_backward(dy, fwd.residual, fwd.mean, fwd.rstd, w, dresidual=dh)
    x64, w64, b64 = (t.double().requires_grad_() for t in (x, w, b))
    h = x64 + r.double()
    d = h - h.mean(1, keepdim=True)
    y = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * w64 + b64
    ((y * dy.double()).sum() + (h * dh.double()).sum()).backward()
    for got, want in ((dx, x64.grad), (dw, w64.grad), (db, b64.grad)):
        assert worst(got, want, 1e-5 * want.abs().mean() + 1e-5 * want.abs()) <= 1

    # central differences along a random direction: step 2^-7, so rounding gives about u / 2^-7 and the
    # third derivative about 2^-14
    def loss(xv, wv, bv):
        f = mbt.tile_layernorm(xv, wv, bv, r, eps=1e-5)
        return ((f.out.double() * dy.double()).sum() + (f.residual.double() * dh.double()).sum()).item()

    e = 2.0 ** -7
    vx, vw, vb = randn((M, N), torch.float32, 36), randn(N, torch.float32, 37), randn(N, torch.float32, 38)
    for got, plus, minus in ((dx.double() * vx.double(), (x + e * vx, w, b), (x - e * vx, w, b)),
                             (dw.double() * vw.double(), (x, w + e * vw, b), (x, w - e * vw, b)),
                             (db.double() * vb.double(), (x, w, b + e * vb), (x, w, b - e * vb))):
        diff = (loss(*plus) - loss(*minus)) / (2 * e)
        assert abs(got.sum().item() - diff) <= 2e-3 * got.square().sum().sqrt().item() + 1e-3 * abs(diff)


@pytest.mark.parametrize("M,N", [(513, 2048), (1500, 8192)])
def test_equal_calls_give_equal_bits_and_graph_capture(M, N):
    x, w, b, dy = (randn(s, torch.bfloat16, 40 + k) for k, s in enumerate(((M, N), N, N, (M, N))))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fwd = mbt.tile_layernorm(x, w, b, stream=s)
    grads = mbt.tile_layernorm_backward(dy, x, fwd.mean, fwd.rstd, w, stream=s)
    s.synchronize()
    first = (fwd.out, fwd.mean, fwd.rstd, *grads)
    again = [torch.zeros_like(t) for t in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mbt.tile_layernorm(x, w, b, out=again[0], mean=again[1], rstd=again[2])
        mbt.tile_layernorm_backward(dy, x, again[1], again[2], w, dx=again[3], dweight=again[4], dbias=again[5])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for p, q in zip(first, again):
        assert torch.equal(p, q)
    assert mbt.tile_status()[0] == 0


def test_past_four_gib():
    """Rows whose offsets pass 32 bits, in elements and in bytes."""
    M, N = 70000, 65536 - 8
    x = torch.ones(1, 1, dtype=torch.float16, device="cuda").expand(M, N).contiguous()
    x[-1] = randn((1, N), torch.float16, 43)[0]
    out = torch.empty_like(x)
    got = mbt.tile_layernorm(x, out=out, eps=1e-6)
    check_forward(x[-3:], None, None, None, mbt.LayerNorm(out[-3:], None, None, got.mean[-3:], got.rstd[-3:]), 1e-6, 0.0, None)
    del x, out, got
    torch.cuda.empty_cache()


def test_refusals():
    x, w = randn((4, 64), torch.float16, 50), randn(64, torch.float16, 51)
    ok = mbt.tile_layernorm(x, w, w)
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(weight=w[:-1]), dict(weight=None),
                dict(weight=w.double()), dict(bias=w.float()), dict(bias=w[1:]), dict(residual=x[:2]), dict(residual=x.float()),
                dict(quant=16), dict(residual_out=x), dict(scales=ok.rstd), dict(out=x.float()), dict(rstd=ok.rstd[:2]),
                dict(mean=ok.mean.half()), dict(quant=0, out=x), dict(quant=0, scales=ok.rstd)):
        with pytest.raises(ValueError):
            mbt.tile_layernorm(**({"x": x, "weight": w, "bias": w} | bad))
    with pytest.raises(mbt.MbtError):
        mbt.tile_layernorm(x, w, eps=-1.0)
    for bad in (dict(dy=x[:2]), dict(dy=x.float()), dict(mean=ok.mean[1:]), dict(rstd=ok.rstd.half()), dict(weight=w[1:]),
                dict(dresidual=x.t()), dict(dx=x.float()), dict(dweight=w), dict(dbias=w)):
        with pytest.raises(ValueError):
            mbt.tile_layernorm_backward(**({"dy": x, "h": x, "mean": ok.mean, "rstd": ok.rstd, "weight": w} | bad))


@pytest.mark.parametrize("N", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 4])
def test_narrow_matrices(N, dtype, pad):
    """Rows shorter than 16 bytes, several of which end in the matrix's last chunk."""
    dt = TYPES[dtype]
    for M in (1, 2, 3, 4, 5, 8, 9, 500, 4001):
        dy, h, d = (pitched(randn((M, N), dt, 97 + k), pad * (k + 1)) for k in range(3))
        w = randn(N, dt, 77)
        fwd = mbt.tile_layernorm(h, w, w, eps=1e-2)
        check_forward(h, w, w, None, fwd, 1e-2, 0.0, None)
        store = torch.full((M * (N + pad) + 64,), 7.0, dtype=dt, device="cuda")
        dx = store[:M * (N + pad)].view(M, N + pad)[:, :N]
        got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, dresidual=d, dx=dx)
        check_backward(dy, h, fwd.mean, fwd.rstd, w, d, *got)
        dx.fill_(7.0)
        assert bool((store == 7).all())
    assert mbt.tile_status()[0] == 0


def test_given_results_raise_their_version():
    x, w = randn((4, 64), torch.float32, 95), randn(64, torch.float32, 96)
    out, ro, mean, rstd, dx, dw, db = (torch.empty_like(x), x.clone(), torch.empty(4, device="cuda"), torch.empty(4, device="cuda"),
                                       torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
    written = (out, ro, mean, rstd, dx, dw, db)
    before = [t._version for t in written]
    mbt.tile_layernorm(x, w, w, x, out=out, residual_out=ro, mean=mean, rstd=rstd)
    mbt.tile_layernorm_backward(x, ro, mean, rstd, w, dx=dx, dweight=dw, dbias=db)
    assert [t._version for t in written] == [b + 1 for b in before]


@pytest.mark.parametrize("M,N,quant", [(1, 64, None), (1, 4096, 0), (5, 1000, 64), (33, 128, 32), (0, 64, 0)])
def test_results_of_one_allocation(M, N, quant):
    """New statistics and scales are ordinary tensors that do not overlap, whatever is given and whatever is not."""
    x = randn((M, N), torch.bfloat16, 110)
    got = mbt.tile_layernorm(x, quant=quant)
    small = [t for t in (got.scales, got.mean, got.rstd) if t is not None]
    spans = sorted((t.data_ptr(), t.data_ptr() + 4 * t.numel()) for t in small)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(t.is_contiguous() for t in small)
    copies = [t.clone() for t in small]
    for k, t in enumerate(small):
        t.add_(1)                                     # one at a time: the others keep their values
        for o, c in zip(small, copies):
            assert o is t or torch.equal(o, c)
        t.copy_(copies[k])                            # (1 added and taken away again would leave a rounding)
    assert [t._version for t in small] == [small[0]._version] * len(small)
    mean = torch.empty(M, device="cuda")
    again = mbt.tile_layernorm(x, quant=quant, mean=mean)
    assert again.mean.data_ptr() == mean.data_ptr() and torch.equal(again.rstd, mbt.tile_layernorm(x, quant=quant).rstd)
    with torch.inference_mode():
        assert torch.equal(mbt.tile_layernorm(x, quant=quant).rstd, again.rstd)
    n = mbt.tile_grad_norm([x])
    n.scale.fill_(3.0)
    assert torch.equal(n.norm, mbt.tile_grad_norm([x]).norm) and n.norm.shape == n.scale.shape == ()


@pytest.mark.parametrize("M,N", [(700, 16384), (2600, 4096), (3001, 1001), (600, 12000)])
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_many_rows_with_an_offset(M, N, dtype, wdt):
    """weight + weight_offset in fp32, whatever the weight's type (zero-centred weights)."""
    dt = TYPES[dtype]
    x, dy = randn((M, N), dt, 120) + 1, randn((M, N), dt, 121)
    w, b = randn(N, TYPES[wdt], 122, 0.01), randn(N, TYPES[wdt], 123)
    got = mbt.tile_layernorm(x, w, b, eps=1e-5, weight_offset=1.0)
    check_forward(x, w, b, None, got, 1e-5, 1.0, None)
    grads = mbt.tile_layernorm_backward(dy, x, got.mean, got.rstd, w, weight_offset=1.0)
    check_backward(dy, x, got.mean, got.rstd, w, None, *grads, 1.0)
    q = mbt.tile_layernorm(x, w, b, eps=1e-5, weight_offset=1.0, quant=0)
    check_forward(x, w, b, None, q, 1e-5, 1.0, 0)
    none = mbt.tile_layernorm(x, None, eps=1e-5, weight_offset=1.0)      # (no weight: no offset)
    check_forward(x, None, None, None, none, 1e-5, 0.0, None)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("scale,eps", [(1e12, 1e-6), (1e17, 1e-6), (1e-15, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,offset", [(64, 4096, 0), (64, 4096, 1), (2000, 1000, 0), (700, 16384, 0)])
def test_any_magnitude(scale, eps, dtype, M, N, offset):
    """Large and small rows, with dy along h so that the projection counts."""
    dt = TYPES[dtype]
    n = randn((M, N), torch.float32, 124).clamp(-3, 3)
    h, w = pitched((n * scale).to(dt), 0, offset), 1 + randn(N, torch.float32, 125, 0.2)
    dy = (0.7 * n + randn((M, N), torch.float32, 126, 0.5)).to(dt)
    fwd = mbt.tile_layernorm(h, w, None, eps=eps)
    check_forward(h, w, None, None, fwd, eps, 0.0, None)
    got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w)
    check_backward(dy, h, fwd.mean, fwd.rstd, w, None, *got)


@pytest.mark.parametrize("M,N,pad", [(300, 24576, 0), (41, 32768, 0), (300, 20001, 7), (33, 17000, 8), (2, 32760, 0), (70, 40000, 0),
                                     (1, 20000, 0), (100, 24001, 0)])
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", None)])
@pytest.mark.parametrize("dres", [False, True])
def test_long_rows_backward(M, N, pad, dtype, wdt, dres):
    """Rows too long for the ring: by chunks where they begin at one, and by elements."""
    dt = TYPES[dtype]
    h, dy = pitched(randn((M, N), dt, 130) + 1, pad), pitched(randn((M, N), dt, 131), pad)
    w = None if wdt is None else randn(N, TYPES[wdt], 132)
    d = pitched(randn((M, N), dt, 133), pad) if dres else None
    fwd = mbt.tile_layernorm(h, w)
    given = dict(dweight=torch.empty(N, device="cuda"), dbias=torch.empty(N, device="cuda"))
    wide = torch.zeros(M, N + pad, dtype=dt, device="cuda")
    got = mbt.tile_layernorm_backward(dy, h, fwd.mean, fwd.rstd, w, dresidual=d, dx=wide[:, :N], **given)
    check_backward(dy, h, fwd.mean, fwd.rstd, w, d, *got)
    assert bool((wide[:, N:] == 0).all())
    copy = dy.contiguous().clone()
    again = mbt.tile_layernorm_backward(copy, h, fwd.mean, fwd.rstd, w, dresidual=d, dx=copy)
    assert pad or torch.equal(again[0], got[0])

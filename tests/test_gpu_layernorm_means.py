"""tile_layernorm on rows that vary little about a large mean, through each of its kernels.

The kernels sum the row, take deviations from the rounded mean m and correct by the
deviations' own mean s.  With u = 2^-24, c = chain(N) + 3 additions and roundings a term of a
sum goes through, A = mean|h| and V = mean|h - mean|:
  m is off by at most D = c u A;
  a deviation is rounded by at most u (|h - mean| + D), so s is off by at most E = c u (V + D);
  the mean m + s is off by E + u |mean|;
  a deviation less s by E + 3 u (|h - mean| + D) (the deviation, s rstd, their sum);
  the variance, sum d^2 / N - s^2, by (c + 3) u (var + D^2) + 2 D E; rstd, relative to itself, by
  half of that over var + eps, and 6 u (the root's reciprocal to two units in the last place).
That is of the size of the rounding of the row's elements, where D alone would be chain(N)
times as much."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import E4M3, OUT_U, TINY, TYPES, U, chain, pitched, randn, worst

pytestmark = pytest.mark.gpu

# few rows in registers; the ring with whole chunks and parts, rows in registers and in their stage
SIZES = [(12, 1000), (12, 4096), (12, 5000), (12, 9001), (12, 16384), (1800, 1000), (1800, 4096), (900, 5001),
         (700, 9001), (400, 16384), (400, 16381)]


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def rows(M, N):
    """fp32: constant rows of values with full significands, and rows that vary little about a mean."""
    x = torch.empty(M, N, device="cuda")
    for k, v in enumerate((1000.1, 12345.678, 0.1, -777777.7)):
        x[k::6] = v
    noise = randn((M, N), torch.float32, 1).double()
    x[4::6] = (1e4 + 1e-2 * noise[4::6]).float()
    x[5::6] = (-1e5 + 0.5 * noise[5::6]).float()
    return x


def check(x, w, b, r, got, eps):
    N = x.shape[1]
    h = x.double() + (0 if r is None else r.double())
    mean = h.mean(1, keepdim=True)
    d = h - mean
    var = d.square().mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    wide, bias = (1 if w is None else w.double()), (0 if b is None else b.double())
    y = d * rstd * wide + bias
    c = chain(N) + 3
    D = c * U * h.abs().mean(1, keepdim=True)
    E = c * U * (d.abs().mean(1, keepdim=True) + D)
    assert worst(got.mean, mean[:, 0], (E + U * (mean.abs() + E))[:, 0]) <= 1
    rel = ((c + 3) * U * (var + D * D) + 2 * D * E) / (2 * (var + eps)) + 6 * U
    assert worst(got.rstd, rstd[:, 0], (rel * rstd)[:, 0]) <= 1
    err = rstd * (E + 3 * U * (d.abs() + D)) * (wide.abs() if w is not None else 1)
    err = (1 + rel) * err + (rel + 4 * U) * (y - bias).abs() + 2 * U * (y.abs() + (bias.abs() if b is not None else 0))
    t = x.dtype
    assert worst(got.out, y, err + OUT_U[t] * (y.abs() + err) + TINY[t]) <= 1
    if r is not None:
        assert torch.equal(got.residual, h.to(t))


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_fp32(M, N, residual):
    x = rows(M, N)
    r = x.clone() if residual else None                # (the sum is exact)
    w, b = randn(N, torch.float32, 2), randn(N, torch.float32, 3)
    check(x, w, b, r, mbt.tile_layernorm(x, w, b, r, eps=1e-5), 1e-5)
    check(x, None, None, r, mbt.tile_layernorm(x, None, None, r, eps=1e-5), 1e-5)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N,pad,offset", [(12, 4096, 0, 1), (12, 5001, 3, 2), (30, 20000, 0, 0)])
def test_rows_by_elements(M, N, pad, offset):
    """Rows that start anywhere, and rows too long for registers."""
    x = pitched(rows(M, N), pad, offset)
    w = randn(N, torch.float32, 4)
    check(x, w, w, None, mbt.tile_layernorm(x, w, w, eps=1e-5), 1e-5)


@pytest.mark.parametrize("dtype,value,add", [("f16", 1000.5, 0.0), ("f16", 0.1, 0.0), ("bf16", 1000.0, 0.33), ("bf16", -52.0, 0.013)])
@pytest.mark.parametrize("M,N", [(5, 4096), (5, 9001), (3000, 9001), (2000, 20008), (160, 32768), (4000, 2056)])
def test_16_bits(M, N, dtype, value, add):
    """Constant rows whose sum fp32 does not hold, by their own bits or with a residual's."""
    dt = TYPES[dtype]
    x = torch.full((M, N), value, device="cuda").to(dt)
    r = torch.full((M, N), add, device="cuda").to(dt) if add else None
    w, b = torch.ones(N, dtype=dt, device="cuda"), torch.full((N,), 0.25, dtype=dt, device="cuda")
    got = mbt.tile_layernorm(x, w, b, r, eps=1e-5)
    check(x, w, b, r, got, 1e-5)
    assert mbt.tile_status()[0] == 0


@pytest.mark.parametrize("M,N", [(5, 4096), (400, 16384), (1800, 4096), (3, 20000)])
@pytest.mark.parametrize("quant", [0, 128])
def test_e4m3(M, N, quant):
    """A constant row is its bias: the largest code, and the bias's scale."""
    x = torch.full((M, N), 12345.678, device="cuda")
    w, b = torch.ones(N, device="cuda"), torch.full((N,), 0.25, device="cuda")
    got = mbt.tile_layernorm(x, w, b, eps=1e-5, quant=quant)
    assert got.out.dtype == E4M3 and bool((got.out.float() == 448).all())
    # y is off by rstd (E + 3 u D) with rstd = 316, D = (chain + 3) u 12345.7: at most 2e-4
    assert worst(got.scales, torch.full_like(got.scales, 0.25 / 448).double(), 1e-3 * 0.25 / 448) <= 1


@pytest.mark.parametrize("M,N", [(6, 256), (6, 9001), (3000, 1000), (400, 16384)])
def test_rows_that_are_not_finite(M, N):
    """An infinity or an overflow leaves mean and rstd what the definitions make of them; other rows keep theirs."""
    x = randn((M, N), torch.float32, 5)
    before = mbt.tile_layernorm(x, eps=1e-5)
    x[1, N // 2] = float("inf")
    x[2, N - 1] = float("-inf")
    x[3, 0] = float("nan")
    x[4] = 3e38                                        # finite elements whose sum is not
    got = mbt.tile_layernorm(x, eps=1e-5)
    assert got.mean[1].item() == float("inf") and got.mean[2].item() == float("-inf") and bool(got.mean[3].isnan())
    assert got.mean[4].item() == float("inf")
    assert bool(got.rstd[1:4].isnan().all()) and bool(got.out[1:5].isnan().all())
    fine = [0, 5]
    for a, c in zip((got.out, got.mean, got.rstd), (before.out, before.mean, before.rstd)):
        assert torch.equal(a[fine], c[fine])
    # squares past fp32's range: an infinite variance, whatever the shift
    x[0] = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1e27, 3e27)
    big = mbt.tile_layernorm(x, eps=1e-5)
    assert big.rstd[0].item() == 0 and bool((big.out[0] == 0).all())

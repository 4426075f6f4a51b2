"""tile_grad_norm within the bound that its order of additions gives.

A chunk is 256 threads x 8 vectors of 16 bytes, and a launch has 4 CTAs an SM, each with
c = ceil(chunks / (4 SMs)) chunks at most (few chunks: 8 CTAs, at most 2 each).  In fp32 a
square is rounded once and goes through at most 4 additions in its vector's half, one of the
halves and 8 of the vectors, then through one for each of the thread's chunks, of which a sum
ends after 64; all after that is in 64 bits.  The root halves what the 14 + min(c, 64)
roundings leave, and the result is rounded once: ((14 + min(c, 64)) / 2 + 1) u."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import TYPES, U, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def tolerance(grads):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunks = sum(-(-g.numel() * g.element_size() // 32768) for g in grads)
    c = max(2, -(-chunks // (4 * sms)))
    return ((14 + min(c, 64)) / 2 + 1) * U


def check(grads):
    want = sum(p.double().square().sum() for g in grads for p in g.split(1 << 26)).sqrt().item()
    got = mbt.tile_grad_norm(grads, max_norm=1.0)
    assert abs(got.norm.item() - want) <= tolerance(grads) * want
    factor = min(1.0, 1.0 / (want + 1e-6))
    assert abs(got.scale.item() - factor) <= (tolerance(grads) + 4 * U) * factor


@pytest.mark.parametrize("sizes", [[5], [1023], [8192, 16384, 5], [250_000], [5_000_000] * 3, [20_000_001, 3], [100] * 2000,
                                   [40_000_000, 999_999], [300_000_000]], ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_bound(sizes, dtype):
    check([randn(n, TYPES[dtype], 1 + k % 7, 1e-2) for k, n in enumerate(sizes)])


@pytest.mark.parametrize("n,dtype", [(1_200_000_000, "bf16"), (600_000_000, "f32")])
def test_equal_values(n, dtype):
    """Roundings that all go one way, in threads of more than 64 chunks."""
    for value in (0.1, 0.7):
        check([torch.full((n,), value, dtype=TYPES[dtype], device="cuda")])
    torch.cuda.empty_cache()

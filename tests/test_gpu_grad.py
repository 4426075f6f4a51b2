"""tile_grad_norm and tile_clip_grads against the formulas in 64 bits.

Tolerance of the norm: a thread adds the squares of a chunk (at most 16 terms in series,
each with a rounding of its own) and then one sum per chunk; with c chunks to a thread a
term goes through at most c + 18 roundings in fp32, the root halves what they leave, and the
result is rounded once: ((c + 18) / 2 + 1) u."""
import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import TYPES, U, randn, worst

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


def norm64(grads):
    return sum((g.double().square().sum() for g in grads), torch.zeros((), dtype=torch.float64, device="cuda")).sqrt()


def tolerance(grads):
    chunks = sum(g.numel() * g.element_size() // 16384 + 1 for g in grads)
    return ((chunks / (6 * 152) + 1 + 18) / 2 + 1) * U


def check(grads, got, most, gs=1.0):
    want = norm64(grads) * abs(gs)
    tol = tolerance(grads)
    if want.item() > torch.finfo(torch.float32).max:   # (70000 values of 1e37: 2.7e39)
        assert got.norm.item() == float("inf")
    else:
        assert worst(got.norm, want, tol * want + 2.0 ** -149) <= 1
    factor = gs * min(1.0, most / (want.item() + EPS)) if most is not None else gs
    assert abs(got.scale.item() - factor) <= (tol + 4 * U) * abs(factor)


def tensors(sizes, types, seed, scale=1e-3):
    return [randn(n, TYPES[types[k % len(types)]], seed + k, scale) for k, n in enumerate(sizes)]


SIZES = [[1], [7], [8], [9], [1023, 0, 5], [4096], [8192 * 3 + 5], [100] * 33, [1, 2, 3, 1000003], [17] * 1600,
         [20_000_001, 3], [5_000_000] * 9]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f16", "f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("most", [1e-2, 1e6, None])
def test_norm(sizes, types, most):
    grads = tensors(sizes, types, 1)
    got = mbt.tile_grad_norm(grads, max_norm=most)
    check(grads, got, most)
    again = mbt.tile_grad_norm(grads, max_norm=most)
    assert torch.equal(got.norm, again.norm) and torch.equal(got.scale, again.scale)


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("most", [1e-2, 1e6])
def test_clip(sizes, most):
    grads = tensors(sizes, ("bf16", "f32", "f16"), 2)
    before = [g.clone() for g in grads]
    got = mbt.tile_clip_grads(grads, most)
    check(before, got, most)
    for g, b in zip(grads, before):
        assert torch.equal(g, (b.float() * got.scale).to(g.dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_views_of_any_alignment(dtype):
    """Tensors that start and end anywhere in a 16-byte chunk; what lies between them stays."""
    store = randn(40000, TYPES[dtype], 3)
    before = store.clone()
    grads, inside, at = [], torch.zeros_like(store, dtype=torch.bool), 1
    for n in [1, 2, 3, 5, 6, 7, 8, 9, 15, 16, 17, 31, 100, 1025, 8193, 12289]:
        grads.append(store[at:at + n])
        inside[at:at + n] = True
        at += n + 1 + n % 3
    check(grads, mbt.tile_grad_norm(grads, max_norm=0.5), 0.5)
    got = mbt.tile_clip_grads(grads, 0.5)
    want = torch.where(inside, (before.float() * got.scale).to(store.dtype), before)
    assert torch.equal(store, want)


def test_strides():
    """Dense tensors in another order than row-major; others are refused."""
    x = randn((40, 50), torch.float32, 4)
    check([x], mbt.tile_grad_norm([x.t()], max_norm=1.0), 1.0)
    for bad in (x[:, ::2], x[:, :49], x[:1].expand(4, 50)):
        with pytest.raises(ValueError, match="dense"):
            mbt.tile_grad_norm([bad])


@pytest.mark.parametrize("dtype,scales", [("bf16", (1e-30, 1e-20, 1e25, 1e37)), ("f32", (1e-38, 1e-30, 1e-20, 1e18, 1e30, 1e37)),
                                          ("f16", (1e-6, 1e4))])
def test_any_magnitude(dtype, scales):
    for s in scales:
        grads = [(randn(n, torch.float32, 5) * s).to(TYPES[dtype]) for n in (3, 1000, 70000)]
        check(grads, mbt.tile_grad_norm(grads), None)
        # beside ordinary ones
        more = grads + [randn(5000, torch.float32, 6)]
        check(more, mbt.tile_grad_norm(more), None)


def test_zeros_and_nothing():
    z = [torch.zeros(10000, device="cuda"), -torch.zeros(33, device="cuda", dtype=torch.bfloat16)]
    got = mbt.tile_grad_norm(z, max_norm=1.0)
    assert got.norm.item() == 0 and got.scale.item() == 1
    got = mbt.tile_grad_norm([], max_norm=1.0)
    assert got.norm.item() == 0 and got.scale.item() == 1
    got = mbt.tile_clip_grads([torch.empty(0, device="cuda")], 1.0)
    assert got.norm.item() == 0 and got.scale.item() == 1


@pytest.mark.parametrize("at", [0, 4, 50000, 99999])
def test_values_that_are_not_finite(at):
    for dtype in TYPES.values():
        g = randn(100000, dtype, 7)
        g[at] = float("inf")
        got = mbt.tile_grad_norm([g], max_norm=1.0)
        assert got.norm.item() == float("inf") and got.scale.item() == 0
        assert mbt.tile_grad_norm([g]).scale.item() == 1
        g[at] = float("nan")
        got = mbt.tile_grad_norm([g], max_norm=1.0)
        assert got.norm.isnan() and got.scale.isnan()


@pytest.mark.parametrize("gs", [0.25, -3.0, 0.0])
def test_grad_scale(gs):
    grads = tensors([1000, 33], ("f32", "bf16"), 8)
    factor = torch.full((1,), gs, device="cuda")
    for most in (0.01, 1e9, None):
        check(grads, mbt.tile_grad_norm(grads, max_norm=most, grad_scale=factor), most, gs)
    before = [g.clone() for g in grads]
    got = mbt.tile_clip_grads(grads, 0.01, grad_scale=factor)
    for g, b in zip(grads, before):
        assert torch.equal(g, (b.float() * got.scale).to(g.dtype))


def test_factor_for_the_optimiser():
    """The factor given to tile_adamw: the step that clipped gradients take."""
    p = randn(5000, torch.float32, 9)
    g = randn(5000, torch.float32, 10)
    results = []
    for clip in (False, True):
        q, m, v, h = p.clone(), torch.zeros_like(p), torch.zeros_like(p), g.clone()
        state = mbt.AdamwTensors([q], [m], [v])
        if clip:
            mbt.tile_clip_grads([h], 0.5)
            mbt.tile_adamw(state, [h], step=1, lr=0.1)
        else:
            mbt.tile_adamw(state, [h], step=1, lr=0.1, grad_scale=mbt.tile_grad_norm([h], max_norm=0.5).scale)
        results.append((q, m, v))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_given_outputs_refusals_and_versions():
    g = randn(100, torch.float32, 11)
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros((), device="cuda")
    before = g._version, norm._version
    got = mbt.tile_clip_grads([g], 1e-3, norm=norm, scale=scale)
    assert got.norm.data_ptr() == norm.data_ptr() and got.scale.data_ptr() == scale.data_ptr()
    assert g._version > before[0] and norm._version > before[1]
    with pytest.raises(mbt.MbtError):
        mbt.tile_clip_grads([g, g[50:]], 1.0)
    for bad in (dict(norm=torch.zeros(2, device="cuda")), dict(scale=torch.zeros(1)),
                dict(grad_scale=torch.zeros(1, device="cuda", dtype=torch.float64))):
        with pytest.raises(ValueError):
            mbt.tile_grad_norm([g], **bad)
    with pytest.raises(mbt.MbtError):
        mbt.tile_grad_norm([g], max_norm=-1.0)


def test_scalars_within_gradients_are_refused():
    g = randn(100, torch.float32, 15)
    before = g.clone()
    for bad in (dict(scale=g[7:8]), dict(norm=g[99:])):
        with pytest.raises(mbt.MbtError):
            mbt.tile_clip_grads([torch.ones(3, device="cuda"), g], 1e-3, **bad)
    assert torch.equal(g, before)
    # a factor that one of them holds is only read
    scale = torch.ones(1, device="cuda")
    got = mbt.tile_clip_grads([g], 1e-3, grad_scale=g[7:8], scale=scale)
    check([before], got, 1e-3, before[7].item())
    assert torch.equal(g, before * scale)


@pytest.mark.parametrize("factor", [0.5, -2.0])
@pytest.mark.parametrize("sizes", [[1000, 33], [3_000_001, 17]], ids=["cluster", "grid"])
def test_factor_written_where_it_was_read(sizes, factor):
    """One tensor as grad_scale and as scale."""
    grads = tensors(sizes, ("f32", "bf16"), 14)
    before = [g.clone() for g in grads]
    for most in (1e-3, 1e9):
        for g, b in zip(grads, before):
            g.copy_(b)
        scale = torch.full((1,), factor, device="cuda")
        got = mbt.tile_clip_grads(grads, most, grad_scale=scale, scale=scale)
        check(before, got, most, factor)
        for g, b in zip(grads, before):
            assert torch.equal(g, (b.float() * scale).to(g.dtype))


@pytest.mark.parametrize("sizes", [[3000, 70001, 12], [5_000_000, 33, 70001]], ids=["cluster", "grid"])
def test_streams_and_graphs(sizes):
    grads = tensors(sizes, ("f32", "bf16"), 12)
    want = mbt.tile_grad_norm(grads, max_norm=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mbt.tile_grad_norm(grads, max_norm=0.1, stream=side)
    side.synchronize()
    assert torch.equal(got.norm, want.norm)
    capture = torch.cuda.Stream()
    mbt.tile_grad_norm(grads, stream=capture)      # the stream's workspace, before the capture
    capture.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=capture):
        got = mbt.tile_clip_grads(grads, 0.1)
    for _ in range(5):                             # odd and even uses of the tickets, eager calls between
        fresh = [randn(g.shape, torch.float32, 13).to(g.dtype) for g in grads]
        for g, f in zip(grads, fresh):
            g.copy_(f)
        with torch.cuda.stream(capture):
            capture.wait_stream(torch.cuda.default_stream())
            graph.replay()
            eager = mbt.tile_grad_norm(fresh, max_norm=0.1)
        capture.synchronize()
        assert torch.equal(got.norm, eager.norm) and torch.equal(got.scale, eager.scale)
        for g, f in zip(grads, fresh):
            assert torch.equal(g, (f.float() * got.scale).to(g.dtype))


def test_past_four_gib():
    """A tensor of more than 2^32 elements, an odd count from an odd address on."""
    n = (1 << 32) + 12345
    store = torch.ones(1, dtype=torch.bfloat16, device="cuda").expand(n + 2).contiguous()
    g = store[1:-1]
    got = mbt.tile_clip_grads([g], 1.0, eps=0.0)
    assert abs(got.norm.item() / n ** 0.5 - 1) < 1e-6
    v = torch.ones((), device="cuda").mul(got.scale).bfloat16()
    assert bool((g[:1000] == v).all()) and bool((g[-1000:] == v).all()) and bool((g[n // 2:n // 2 + 1000] == v).all())
    assert store[0] == 1 and store[-1] == 1
    assert abs(g.view(-1)[:1 << 31].sum(dtype=torch.float64).item() / (v.double().item() * (1 << 31)) - 1) < 1e-9
    del store, g
    torch.cuda.empty_cache()


def test_long_sums():
    """Some 1700 chunks a thread, whose sums in fp32 alone would drift one way.

    A square is one rounding, its chunk's 32 are at most 10 additions deep, and 64 chunks
    are added before fp32 ends: 75 half steps of the sum, half as many of its root, and one."""
    n, x = 1 << 33, 1.6491228342056274
    g = torch.full((n,), x, device="cuda")
    got = mbt.tile_grad_norm([g])
    assert abs(got.norm.item() / (g[0].double().item() * n ** 0.5) - 1) <= 38.5 * U
    del g
    torch.cuda.empty_cache()

"""tile_adamw against the formulas in 64 bits."""
import math

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from layer_helpers import E4M3, OUT_U, TINY, TYPES, U, e4m3_half_spacing, randn, worst

pytestmark = pytest.mark.gpu
BLOCK = 256


@pytest.fixture(scope="module", autouse=True)
def setup():
    mbt._build.build()
    torch.cuda.set_device(0)


SIZES = [1, 7, 255, 256, 257, 4095, 4096, 4097, 20000, 0, 3, 70001]
HYPER = dict(step=5, lr=2e-3, beta1=0.9, beta2=0.995, eps=1e-8, weight_decay=0.05)


def shifted(t, by):
    store = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
    view = store[by:by + t.numel()]
    view.copy_(t)
    return view


def make(sizes, pdt, gdt, seed, master=False, shift=0):
    w = [randn(n, torch.float32, seed + k, 0.05) for k, n in enumerate(sizes)]
    p = [shifted(x.to(pdt), shift) for x in w]
    g = [shifted(randn(n, gdt, seed + 100 + k, 0.01), shift) for k, n in enumerate(sizes)]
    m = [randn(n, torch.float32, seed + 200 + k, 0.002) for k, n in enumerate(sizes)]
    v = [randn(n, torch.float32, seed + 300 + k, 0.01).square() + 1e-6 for k, n in enumerate(sizes)]
    return p, g, m, v, w if master else None


def step64(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, scale=1.0):
    g = g.double() * scale
    m = beta1 * m.double() + (1 - beta1) * g
    v = beta2 * v.double() + (1 - beta2) * g * g
    update = lr / (1 - beta1 ** step) * m / (v.sqrt() / math.sqrt(1 - beta2 ** step) + eps)
    return p.double() * (1 - lr * weight_decay) - update, m, v, update


def check32(old, new, scale=1.0, **hyper):
    p, g, m, v, w = old
    p2, m2, v2, w2 = new
    for k in range(len(p)):
        base = p[k] if w is None else w[k]
        want, wm, wv, update = step64(base, g[k], m[k], v[k], scale=scale, **hyper)
        gs = g[k].double().abs() * scale
        # m, v: three roundings of each term (and of the betas); the update: of m, v, sqrt and the quotient
        bm = 8 * U * (m[k].double().abs() + gs)
        assert worst(m2[k], wm, bm + 1e-40) <= 1
        assert worst(v2[k], wv, 8 * U * wv + 1e-38) <= 1
        lr_eff = hyper["lr"] / (1 - hyper["beta1"] ** hyper["step"])
        denom = wv.sqrt() / math.sqrt(1 - hyper["beta2"] ** hyper["step"]) + hyper["eps"]
        bp = 4 * U * want.abs() + 4 * U * base.double().abs() + 24 * U * update.abs() + lr_eff * bm / denom
        if w is not None:
            assert worst(w2[k], want, bp) <= 1
        assert worst(p2[k], want, bp + OUT_U[p2[k].dtype] * want.abs() + TINY[p2[k].dtype]) <= 1


@pytest.mark.parametrize("pdt,gdt,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                            ("bf16", "bf16", True), ("bf16", "f32", True), ("f16", "f16", False),
                                            ("f16", "f32", True), ("f16", "bf16", False), ("f32", "f16", False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_states_in_32_bits(pdt, gdt, master, shift):
    p, g, m, v, w = make(SIZES, TYPES[pdt], TYPES[gdt], 1, master, shift)
    if shift:
        m, v = [shifted(t, 1) for t in m], [shifted(t, 3) for t in v]
    old = [[t.clone() for t in x] if x is not None else None for x in (p, g, m, v, w)]
    mbt.tile_adamw(mbt.AdamwTensors(p, m, v, master=w), g, **HYPER)
    check32(old, (p, m, v, w), **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(g, old[1]))


@pytest.mark.parametrize("count", [1, 32, 33, 500, 1000])
def test_many_tensors(count):
    sizes = [1 + 97 * k % 6000 for k in range(count)]
    old = make(sizes, torch.float32, torch.float32, 2)
    p, g, m, v, _ = ([t.clone() for t in x] if x is not None else None for x in old)
    mbt.tile_adamw(mbt.AdamwTensors(p, m, v), g, **HYPER)
    check32(old, (p, m, v, None), **HYPER)


def test_grad_scale_streams_and_graph():
    old = make([5000, 100], torch.float32, torch.float32, 3)
    p, g, m, v, _ = ([t.clone() for t in x] if x is not None else None for x in old)
    scale = torch.tensor(0.25, device="cuda")
    table = mbt.AdamwTensors(p, m, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mbt.tile_adamw(table, g, grad_scale=scale, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    check32(old, (p, m, v, None), scale=0.25, **HYPER)


def test_zero_gradients_and_first_step():
    p = [torch.ones(1000, device="cuda")]
    z = lambda: [torch.zeros(1000, device="cuda")]  # noqa: E731
    m, v = z(), z()
    mbt.tile_adamw(mbt.AdamwTensors(p, m, v), z(), step=1, lr=0.1, weight_decay=0.5)
    assert bool((p[0] == torch.tensor(0.95, device="cuda")).all()) and bool((m[0] == 0).all())
    # the first step moves every weight by lr in the gradient's direction
    p, g = [torch.zeros(1000, device="cuda")], [randn(1000, torch.float32, 4)]
    mbt.tile_adamw(mbt.AdamwTensors(p, z(), z()), g, step=1, lr=0.1, eps=0.0)
    assert worst(p[0], -0.1 * g[0].sign().double(), torch.tensor(0.1 * 32 * U)) <= 1


# 8-bit states ----------------------------------------------------------------------------------------------------

def blocks(t):
    n = t.numel()
    return torch.nn.functional.pad(t, (0, -n % BLOCK)).view(-1, BLOCK)


def to_codes(t):
    b = blocks(t)
    s = (b.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    return (b / s[:, None]).clamp(-448, 448).view(-1)[:t.numel()].to(E4M3), s


def values(code, scale, dtype=torch.float64):
    return (blocks(code.to(dtype)) * scale.to(dtype)[:, None]).view(-1)[:code.numel()]


def random16(n, tensor, seed):
    i = torch.arange(n, device="cuda")
    full = 0xFFFFFFFF
    h = ((tensor * 0x9E3779B9 + i // 2) & full) ^ seed
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & full
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & full
    h = h ^ (h >> 16)
    return torch.where(i % 2 == 1, h >> 16, h & 0xFFFF)


def make8(sizes, pdt, seed, master=False, shift=0):
    p, g, m, v, w = make(sizes, pdt, pdt, seed, master, shift)
    mq = [to_codes(t) for t in m]
    vq = [to_codes(t.sqrt()) for t in v]
    return p, g, [shifted(c, shift) for c, _ in mq], [shifted(c, shift) for c, _ in vq], w, [s for _, s in mq], [s for _, s in vq]


@pytest.mark.parametrize("pdt,master", [("f32", False), ("bf16", False), ("bf16", True), ("f16", False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_states_in_8_bits(pdt, master, shift):
    p, g, m, v, w, ms, vs = make8(SIZES, TYPES[pdt], 5, master, shift)
    old = [[t.clone() for t in x] if x is not None else None for x in (p, g, m, v, w, ms, vs)]
    seed = 12345
    mbt.tile_adamw(mbt.AdamwTensors(p, m, v, master=w, m_scales=ms, v_scales=vs), g, seed=seed, **HYPER)
    p0, g0, m0, v0, w0, ms0, vs0 = old
    m32 = [values(c, s) for c, s in zip(m0, ms0)]
    v32 = [values(c, s).square() for c, s in zip(v0, vs0)]
    for k, n in enumerate(SIZES):
        if n == 0:
            continue
        base = p0[k] if w0 is None else w0[k]
        want, wm, wv, update = step64(base, g0[k], m32[k], v32[k], **HYPER)
        bp = 8 * U * (want.abs() + base.double().abs()) + 64 * U * update.abs()
        bp += HYPER["lr"] * 10 * 8 * U * (m32[k].abs() + g0[k].double().abs()) / wv.sqrt()
        assert worst(p[k], want, bp + OUT_U[p[k].dtype] * want.abs() + TINY[p[k].dtype]) <= 1
        if master:
            assert worst(w[k], want, bp) <= 1
        root = wv.sqrt()
        sm = (blocks(wm).abs().amax(1) / 448).clamp_min(2.0 ** -126)
        sv = (blocks(root).amax(1) / 448).clamp_min(2.0 ** -126)
        assert worst(ms[k], sm, 32 * U * sm) <= 1 and worst(vs[k], sv, 32 * U * sv) <= 1
        tm = (blocks(wm) / sm[:, None]).view(-1)[:n]
        tv = (blocks(root) / sv[:, None]).view(-1)[:n]
        cm, cv = m[k].double(), v[k].double()
        assert worst(cm, tm, e4m3_half_spacing(tm * (1 + 64 * U)) + 64 * U * 448) <= 1
        assert bool(((cv - tv).abs() <= 2 * e4m3_half_spacing(tv * (1 + 64 * U)) * (1 + 64 * U)).all())
        # the codes are those of the stated random bits, but where fp32 rounding moves a value across them
        low = torch.where(tv < 2.0 ** -6, 2.0 ** -6, 0.0)
        bits = (tv.float() + low.float()).view(torch.int32).long() + (random16(n, k, seed) << 4 | 8)
        expect = ((bits & ~0xFFFFF).int().view(torch.float32) - low.float()).clamp(2.0 ** -9, 448.0)
        assert (cv != expect.double()).double().mean().item() <= 2e-3 + (1.5 / n if n < 1000 else 0)


def test_random_rounding_has_no_bias_and_never_stores_zero():
    """beta2 near 1: the mean of sqrt(v) over many seeds is the exact one, though a
    step is far below half a code; tiny entries keep a code above 0."""
    n = BLOCK * 64
    g = [torch.zeros(n, device="cuda")]
    start = torch.rand(n, generator=torch.Generator("cuda").manual_seed(6), device="cuda") * 0.9 + 0.05
    start[::BLOCK] = 1.0
    start[1::BLOCK] = 1e-9
    code, scale = to_codes(start)
    code[1::BLOCK] = torch.tensor(2.0 ** -9, device="cuda").to(E4M3)
    held = values(code, scale)
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    runs = 400
    # blocks with an entry at 0.9995 of its old value beside a larger new one: g lifts entry 0 alone
    g[0][::BLOCK] = 10.0
    for seed in range(runs):
        p, m, ms = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda").to(E4M3)], [torch.zeros(n // BLOCK, device="cuda")]
        v, vs = [code.clone()], [scale.clone()]
        mbt.tile_adamw(mbt.AdamwTensors(p, m, v, m_scales=ms, v_scales=vs), g, step=10, lr=0.0, beta2=0.999, seed=seed * 7919)
        assert bool((v[0].float() > 0).all())
        total += values(v[0], vs[0])
    want = (0.999 * held.square() + 0.001 * g[0].double().square()).sqrt()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::BLOCK] = keep[1::BLOCK] = False
    rel = ((total / runs - want) / want)[keep]
    # a code is within 1/8 of its value: the mean of `runs` draws of 16320 entries is off by at most
    # 1/8 / 2 / sqrt(runs * 16128) = 2.5e-5 (one sigma); nearest rounding would be off by up to 1/16
    assert abs(rel.mean().item()) <= 1.5e-4
    assert rel.abs().max().item() <= 0.0625 / math.sqrt(runs) * 6


def test_refusals():
    f = lambda n=8, dt=torch.float32: [torch.zeros(n, dtype=dt, device="cuda")]  # noqa: E731
    e = lambda: f(8, E4M3)  # noqa: E731
    for bad in (lambda: mbt.AdamwTensors(f(), f(), f() + f()), lambda: mbt.AdamwTensors(f(), f(9), f()),
                lambda: mbt.AdamwTensors(f(), f(8, torch.float16), f()), lambda: mbt.AdamwTensors(f(), e(), e()),
                lambda: mbt.AdamwTensors(f(), f(), f(), master=f()), lambda: mbt.AdamwTensors([f()[0].cpu()], f(), f()),
                lambda: mbt.AdamwTensors(f(), e(), e(), m_scales=f(2), v_scales=f(1)),
                lambda: mbt.AdamwTensors([f()[0][::2]], f(4), f(4))):
        with pytest.raises(ValueError):
            bad()
    table = mbt.AdamwTensors(f(), f(), f())
    for g in ([], f(9), f(8, torch.float64), [f()[0].cpu()], [f(16)[0][::2]]):
        with pytest.raises(ValueError):
            mbt.tile_adamw(table, g, step=1, lr=1e-3)
    for bad in (dict(step=0), dict(lr=-1.0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(weight_decay=-1.0)):
        with pytest.raises(mbt.MbtError) as err:
            mbt.tile_adamw(table, f(), **({"step": 1, "lr": 1e-3} | bad))
        assert err.value.code == -1
    mbt.tile_adamw(mbt.AdamwTensors([], [], []), [], step=1, lr=1e-3)


@pytest.mark.parametrize("size", [1e-18, 1e-19, 1e-20])
@pytest.mark.parametrize("shift", [0, 1])
def test_8_bit_states_of_tiny_gradients(size, shift):
    """v below fp32's normal range: its root is the update's divisor (eps = 0) and the stored code."""
    n, lr, seed = 4096 + 100, 0.1, 77
    g = shifted((0.5 + randn(n, torch.float32, 90).abs().clamp_max(1)) * randn(n, torch.float32, 91).sign() * size, shift)
    z = lambda k, dt=torch.float32: [torch.zeros(k, device="cuda").to(dt)]  # noqa: E731
    p, m, v, ms, vs = z(n), z(n, E4M3), z(n, E4M3), z(-(-n // BLOCK)), z(-(-n // BLOCK))
    mbt.tile_adamw(mbt.AdamwTensors(p, m, v, m_scales=ms, v_scales=vs), [g], step=1, lr=lr, eps=0.0, seed=seed)
    root = (g * 0.001 * g).double().sqrt()    # (v as fp32 holds it)
    assert bool((root > 0).all()) and float(root.max()) < 2.0 ** -63
    want = -lr * g.double() / (root / math.sqrt(0.001))
    assert worst(p[0], want, 64 * U * want.abs()) <= 1
    scale = blocks(root).amax(1) / 448
    assert worst(vs[0], scale, 4 * U * scale) <= 1
    t = (blocks(root) / scale[:, None]).view(-1)[:n]
    # rounded up or down: within one spacing
    assert worst(v[0].float(), t, 2 * e4m3_half_spacing(t * (1 + 64 * U)) * (1 + 64 * U)) <= 1


def test_replaced_data_are_refused():
    """A parameter or state whose data were replaced: an error, and nothing written where they lay."""
    make_ = lambda: [torch.ones(100, device="cuda") for _ in range(3)]  # noqa: E731
    g = [torch.ones(100, device="cuda")]
    for k in range(3):
        t = make_()
        table = mbt.AdamwTensors([t[0]], [t[1]], [t[2]])
        old = t[k].detach()
        t[k].data = torch.full((100,), 2.0, device="cuda")
        with pytest.raises(ValueError, match="other data"):
            mbt.tile_adamw(table, g, step=1, lr=0.1)
        assert bool((old == 1).all()) and all(bool((x == (2 if i == k else 1)).all()) for i, x in enumerate(t))
        mbt.tile_adamw(mbt.AdamwTensors([t[0]], [t[1]], [t[2]]), g, step=1, lr=0.1)
        assert bool((t[k] != 2).all())

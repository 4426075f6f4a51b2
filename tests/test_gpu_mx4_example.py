"""The layer-normed 4-bit linear layer: that it runs, and its gradients and update against the formulas."""
import os
import sys

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from conftest import ROOT
from layer_helpers import randn
from mx4_helpers import untile_scales, values64

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_runs():
    import mx4_linear

    r = mx4_linear.main(steps=8)
    assert all(torch.isfinite(torch.tensor(v)) for v in r.values())
    # 4-bit rounding of both operands: an element is off by at most half its code's spacing, a quarter of its value
    # beside the smallest codes; products of independent errors stay below that
    assert 0 < r["served_difference"] < 0.5


def values(m):
    rows, K = m.q.shape[0], 2 * m.q.shape[1]
    return values64(m.q, untile_scales(m.scales, rows, K // m.block), m.block, m.tensor_scale)


@pytest.mark.parametrize("tokens,width,outputs", [(64, 256, 96), (200, 1024, 130)])
def test_a_step_against_the_formulas(tokens, width, outputs):
    """One training step: forward, gradients (straight through the roundings), norm, clipped update, in 64 bits.

    Tolerances: bf16 results carry 2^-8 of their magnitude each; products of bf16 values of K terms are summed in
    fp32 and rounded once, so a gradient is off by 2^-8 for its own rounding and as much for each bf16 factor that
    was rounded before it (d, d_norm, the dequantised operands)."""
    import mx4_linear as ex

    layer = ex.Layer(randn((outputs, width), torch.bfloat16, 1, 0.05), 1 + randn(width, torch.bfloat16, 2, 0.2),
                     randn(width, torch.bfloat16, 3, 0.1))
    x, residual = randn((tokens, width), torch.bfloat16, 4), randn((tokens, width), torch.bfloat16, 5)
    d = randn((tokens, outputs), torch.bfloat16, 6, 0.1)
    f = ex.forward(layer, x, residual)
    a, w = values(f.rounded), values(f.weight)
    out = a @ w.t()
    assert ((f.out.double() - out).norm() / out.norm()).item() < 1e-5
    dx, (dw, dg, db) = ex.backward(layer, f, d)
    h = f.norm.residual.double()
    xh = (h - h.mean(1, keepdim=True)) / (h.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    d_norm = d.double() @ w
    g = d_norm * layer.gain.double()
    want_dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) / (h.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    for got, want in ((dw, d.double().t() @ a), (dg, (d_norm * xh).sum(0)), (db, d_norm.sum(0)), (dx, want_dx)):
        assert ((got.double() - want).norm() / want.norm()).item() < 4 * 2.0 ** -8
    # the clipped step
    grads = (dw, dg, db)
    total = mbt.tile_grad_norm(grads, max_norm=0.1)
    norm = sum(t.double().square().sum() for t in grads).sqrt()
    assert abs(total.norm.item() / norm.item() - 1) < 1e-5
    params = [p.clone() for p in layer]
    masters = [p.float() for p in params]
    moments = [[torch.zeros_like(p) for p in masters] for _ in range(2)]
    mbt.tile_adamw(mbt.AdamwTensors(params, *moments, master=masters), grads, step=1, lr=1e-2, eps=1e-3,
                   grad_scale=total.scale)
    for p, q, t in zip(layer, masters, grads):
        s = t.double() * min(1.0, 0.1 / (norm.item() + 1e-6))
        want = p.double() - 1e-2 * s / (s.abs() + 1e-3)     # (m / bc1 = s, sqrt(v / bc2) = |s| after one step)
        assert (q.double() - want).abs().max().item() < 1e-2 * 1e-4
    assert mbt.tile_status()[0] == 0

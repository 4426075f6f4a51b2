"""A layer-normed linear layer trained with 4-bit floating-point products.

    python examples/mx4_linear.py [--steps 60]

The layer is y = layernorm(x + residual) @ W^T.  Forward, both operands of the product are
rounded to microscaled 4-bit floats (``tile_mx4_quantize``, ``tile_mx4_matmul``); W itself
is kept in bf16.  Backward, the roundings count as the identity: the gradients of W and of
the norm's output are products with the rounded operands' values (torch's, on what
``tile_mx4_dequantize`` gives), ``tile_layernorm_backward`` takes the second on to the norm.
``tile_grad_norm`` finds the norm of all gradients and the factor that clips it, which
``tile_adamw`` takes as ``grad_scale``.  Served token by token, W is rounded once.
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mbarrier_async_tile_gb300 as mbt  # noqa: E402

SCALE_TIMES_CODE = 448.0 * 6.0   # the largest scale times the largest code


def to_mx4(x: torch.Tensor) -> mbt.Mx4:
    """x in blocks of 16, its scales relative to its largest magnitude."""
    largest = x.abs().amax().float().clamp_min(1e-12)
    return mbt.tile_mx4_quantize(x, tensor_scale=(largest / SCALE_TIMES_CODE).view(1))


class Layer(NamedTuple):
    weight: torch.Tensor         # outputs x width, bf16
    gain: torch.Tensor           # the norm's weight and bias, bf16
    bias: torch.Tensor


class Forward(NamedTuple):
    out: torch.Tensor
    norm: mbt.LayerNorm
    rounded: mbt.Mx4             # the norm's output
    weight: mbt.Mx4


def forward(layer: Layer, x: torch.Tensor, residual: torch.Tensor) -> Forward:
    norm = mbt.tile_layernorm(x, layer.gain, layer.bias, residual)
    rounded, weight = to_mx4(norm.out), to_mx4(layer.weight)
    return Forward(mbt.tile_mx4_matmul(rounded, weight, out_dtype=torch.float32), norm, rounded, weight)


def backward(layer: Layer, f: Forward, d: torch.Tensor):
    """Gradients (of x and residual alike, of weight, gain and bias) from out's, in bf16."""
    d_weight = d.t() @ mbt.tile_mx4_dequantize(f.rounded)
    d_norm = d @ mbt.tile_mx4_dequantize(f.weight)
    dx, d_gain, d_bias = mbt.tile_layernorm_backward(d_norm, f.norm.residual, f.norm.mean, f.norm.rstd, layer.gain)
    return dx, (d_weight, d_gain.to(torch.bfloat16), d_bias.to(torch.bfloat16))


def main(steps: int = 60, tokens: int = 1024, width: int = 1024, outputs: int = 512, seed: int = 0) -> dict:
    mbt._build.build()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    target = randn(outputs, width, scale=width ** -0.5)
    layer = Layer(randn(outputs, width, scale=0.02), torch.ones(width, dtype=torch.bfloat16, device="cuda"),
                  torch.zeros(width, dtype=torch.bfloat16, device="cuda"))
    masters = [p.float() for p in layer]
    moments = [[torch.zeros_like(p) for p in masters] for _ in range(2)]
    optimiser = mbt.AdamwTensors(list(layer), *moments, master=masters)
    losses, norms = [], []
    for step in range(1, steps + 1):
        x, residual = randn(tokens, width), randn(tokens, width)
        f = forward(layer, x, residual)
        err = f.out - (f.norm.out @ target.t()).float()
        losses.append(err.square().mean())
        _, grads = backward(layer, f, (err * (2 / outputs)).bfloat16())   # (scaled up by the tokens' count)
        total = mbt.tile_grad_norm(grads, max_norm=1.0, grad_scale=torch.full((1,), 1 / tokens, device="cuda"))
        norms.append(total.norm)
        mbt.tile_adamw(optimiser, grads, step=step, lr=3e-3, grad_scale=total.scale)
    weight = to_mx4(layer.weight)
    worst = 0.0
    for _ in range(4):   # one token at a time
        x, residual = randn(1, width), randn(1, width)
        n = mbt.tile_layernorm(x, layer.gain, layer.bias, residual)
        served = mbt.tile_mx4_matmul(to_mx4(n.out), weight)
        want = n.out @ layer.weight.t()
        worst = max(worst, ((served - want).float().norm() / want.float().norm()).item())
    code, info = mbt.tile_status()
    assert code == 0, info
    result = {"first_loss": losses[0].item(), "last_loss": losses[-1].item(), "last_norm": norms[-1].item(),
              "served_difference": worst}
    print(f"loss {result['first_loss']:.4f} -> {result['last_loss']:.4f} in {steps} steps; "
          f"tokens served from 4-bit floats differ from bf16 by {100 * worst:.1f} %")
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)

"""The layer operators together: train a normed linear layer, then serve it in 4 bits.

    python examples/norm_linear.py [--steps 60]

The layer is y = norm(x + residual) @ W^T.  Training: ``tile_rmsnorm`` forward,
``tile_rmsnorm_backward``, ``tile_adamw`` on W and the norm's weight with both
states in 8 bits (the matrix products are torch's).  Serving: W laid out once in
4 bits, then, token by token, ``tile_rmsnorm`` with an e4m3 output and
``tile_w4_matvec`` on its codes and scales.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mbarrier_async_tile_gb300 as mbt  # noqa: E402

BLOCK = 256   # elements of an 8-bit optimiser state that share a scale


def to_4_bits(weight: torch.Tensor, group: int = 128):
    """(q, scales, zeros) of a matrix: each group of a row between its least and
    largest value in 15 steps."""
    N, K = weight.shape
    w = weight.float().view(N, K // group, group)
    low, high = w.amin(2).clamp_max(0), w.amax(2).clamp_min(0)
    scales = ((high - low) / 15).clamp_min(1e-8).to(torch.bfloat16)
    s = scales.float()[:, :, None]
    zeros = (-low[:, :, None] / s).round().clamp(0, 15)
    q = ((w / s).round() + zeros).clamp(0, 15).to(torch.uint8).view(N, K)
    return q[:, 0::2] | q[:, 1::2] << 4, scales, zeros[:, :, 0].to(torch.uint8)


def state8(p: torch.Tensor):
    """A zero 8-bit state and its scales."""
    return (torch.zeros(p.shape, device=p.device).to(mbt.E4M3),
            torch.zeros(-(-p.numel() // BLOCK), device=p.device))


def main(steps: int = 60, tokens: int = 1024, width: int = 1024, outputs: int = 512, seed: int = 0) -> dict:
    mbt._build.build()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    target = randn(outputs, width, scale=width ** -0.5)
    weight, norm_weight = randn(outputs, width, scale=0.02), torch.ones(width, dtype=torch.bfloat16, device="cuda")
    (m1, ms1), (v1, vs1), (m2, ms2), (v2, vs2) = (state8(p) for p in (weight, weight, norm_weight, norm_weight))
    optimiser = mbt.AdamwTensors([weight, norm_weight], [m1, m2], [v1, v2], m_scales=[ms1, ms2], v_scales=[vs1, vs2])
    losses = []
    for step in range(1, steps + 1):
        x, residual = randn(tokens, width), randn(tokens, width)
        fwd = mbt.tile_rmsnorm(x, norm_weight, residual)
        err = (fwd.out @ weight.t() - fwd.out @ target.t()).float()
        losses.append(err.square().mean())
        d = (err * (2 / err.numel())).bfloat16()
        grad_w = d.t() @ fwd.out
        _, grad_norm = mbt.tile_rmsnorm_backward(d @ weight, fwd.residual, fwd.rstd, norm_weight)
        mbt.tile_adamw(optimiser, [grad_w, grad_norm.bfloat16()], step=step, lr=3e-3, weight_decay=0.0, seed=step)
    q, scales, zeros = to_4_bits(weight)
    worst = 0.0
    for _ in range(4):   # one token at a time
        x, residual = randn(1, width), randn(1, width)
        n = mbt.tile_rmsnorm(x, norm_weight, residual, quant=128)
        served = mbt.tile_w4_matvec(n.out, q, scales, zeros, group=128, x_scales=n.scales)
        want = mbt.tile_rmsnorm(x, norm_weight, residual).out @ weight.t()
        worst = max(worst, ((served - want).float().norm() / want.float().norm()).item())
    code, info = mbt.tile_status()
    assert code == 0, info
    result = {"first_loss": losses[0].item(), "last_loss": losses[-1].item(), "served_difference": worst}
    print(f"loss {result['first_loss']:.4f} -> {result['last_loss']:.4f} in {steps} steps; "
          f"tokens served from 4-bit weights and 8-bit activations differ by {100 * worst:.1f} %")
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)

"""Plain 64-bit forms and error bounds shared by the layer operators' tests.

u = 2^-24 is fp32's unit roundoff.  A result that is a sum of n terms has an
error of at most (chain length) u times the sum of the terms' magnitudes, where
the chain is the longest run of additions one term goes through.
"""
import torch

U = 2.0 ** -24
OUT_U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}
# spacing of the type's subnormal values: the absolute error of a tiny result
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}
E4M3 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def pitched(t, pad, offset=0):
    """The values of `t` in rows `pad` elements longer, `offset` elements into a NaN-filled storage."""
    M, N = t.shape
    store = torch.full((M * (N + pad) + offset + 64,), float("nan"), device=t.device).to(t.dtype)
    view = store[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(t)
    return view


def chain(n):
    """Additions a term of a row's sum goes through: at least 512 partial sums, then a tree."""
    return n / 512 + 40


def worst(got, want, bound):
    """Largest |got - want| / bound."""
    err = (got.double() - want).abs()
    return (err / bound).max().item() if err.numel() else 0.0


def norm64(x, w, r, eps, offset):
    h = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / (h.square().mean(1) + eps).sqrt()
    return h, rstd, h * rstd[:, None] * (1 if w is None else w.double() + offset)


def e4m3_half_spacing(t):
    """Half the distance between e4m3 neighbours at magnitude |t|."""
    e = t.abs().clamp_min(2.0 ** -6).log2().floor()
    return 2.0 ** (e - 4)

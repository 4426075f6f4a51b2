"""Python binding of the layer operators: RMS norm, layer norm and their gradients, the
4-bit matrix-vector product, matrices in 4-bit floats and their product, the
gradients' norm, the AdamW step (see include/mbtile.h).

The signatures and documentation; checks, allocation of results that the caller
does not provide, and the call are compiled (csrc/mbtile_torch.cpp).  If the
compiled parts are missing, every call raises; there is no fallback path.

New results of at most 64 KiB of one call of layer norm, its gradient, the gradients'
norm or the quantisation to 4-bit floats are parts of one storage: values and versions
are each tensor's own, but saving one with ``torch.save`` writes the whole storage, one
that is kept keeps the memory of all, and a storage that is resized or freed takes the
others with it.  Results that the caller gives have storages of their own.

Autograd sees none of the operators: results carry no gradient, whatever the
inputs require (the gradient of the norm is a call of its own).  It is told which
of the caller's tensors a call has written: a graph that saved one of them before
raises in its backward pass.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
from typing import NamedTuple

import torch

from . import DTYPE_CODE, MbtError, _build, _load

E4M3 = torch.float8_e4m3fn
MBT_E4M3 = 3
ADAMW_BLOCK = 256
_CODE = {**DTYPE_CODE, E4M3: MBT_E4M3}
_QUANT = {None: -1, 0: 0, 32: 32, 64: 64, 128: 128}

_compiled = None


def _ext():
    """The compiled half of the binding, loaded on first use."""
    global _compiled
    if _compiled is None:
        _load()
        path = _build.require_binding()
        loader = importlib.machinery.ExtensionFileLoader("_mbtile_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mbtile_torch", loader))
        loader.exec_module(module)
        module.set_error(MbtError)
        _compiled = module
    return _compiled


def _call(function: str, stream, *args):
    """A compiled call on `stream`, where its results are allocated too (None: the current one)."""
    if stream is None:
        return getattr(_compiled or _ext(), function)(*args)
    with torch.cuda.stream(stream):
        return getattr(_compiled or _ext(), function)(*args)


def _dense(t: torch.Tensor, name: str, shape, dtypes, device: torch.device) -> int:
    """Address of a dense tensor that must have this shape and one of the types."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)} and type "
                         f"{' or '.join(str(d) for d in dtypes)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}")
    return t.data_ptr()


_F32 = (torch.float32,)


class RmsNorm(NamedTuple):
    """Results of :func:`tile_rmsnorm`; ``scales`` and ``residual`` may be None."""
    out: torch.Tensor
    scales: torch.Tensor | None
    residual: torch.Tensor | None
    rstd: torch.Tensor


def tile_rmsnorm(x: torch.Tensor, weight: torch.Tensor | None = None,
                 residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                 weight_offset: float = 0.0, quant: int | None = None,
                 out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                 residual_out: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                 stream=None) -> RmsNorm:
    """h = x + residual; out = h / sqrt(mean(h^2) + eps) * (weight + weight_offset), row by row.

    ``x``, ``residual``, ``residual_out``: M x N CUDA matrices of one type (fp16,
    bf16, fp32) with unit column stride; ``weight``: N elements of any of the
    three.  ``quant``: None for ``out`` in x's type; 0 for e4m3 with one fp32
    scale a row (``scales``: M x 1); 32, 64 or 128 for one per that many columns
    (``scales``: M x ceil(N / quant)).  ``residual_out`` receives h (allocated
    if there is a residual) and may be ``residual`` itself.  ``rstd``: fp32[M]
    for :func:`tile_rmsnorm_backward`."""
    if quant not in _QUANT:
        raise ValueError("quant must be None, 0, 32, 64 or 128")
    return RmsNorm(*_call("rmsnorm", stream, x, weight, residual, eps, weight_offset, _QUANT[quant], out, scales,
                          residual_out, rstd))


def tile_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                          weight: torch.Tensor | None = None, *,
                          dresidual: torch.Tensor | None = None, weight_offset: float = 0.0,
                          dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                          stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradient of :func:`tile_rmsnorm` at ``h`` (its ``residual``, or x without
    one): ``(dx, dweight)``, dx in h's type and the gradient of x and residual
    alike, dweight fp32[N] (None without a weight, unless a ``dweight`` to write
    is given).  ``dresidual``: the gradient that reaches h past the norm, added
    to dx.  ``dx`` may be ``dy`` or ``dresidual`` itself."""
    return _call("rmsnorm_backward", stream, dy, h, rstd, weight, dresidual, weight_offset, dx, dweight)


class LayerNorm(NamedTuple):
    """Results of :func:`tile_layernorm`; ``scales`` and ``residual`` may be None."""
    out: torch.Tensor
    scales: torch.Tensor | None
    residual: torch.Tensor | None
    mean: torch.Tensor
    rstd: torch.Tensor


def tile_layernorm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   residual: torch.Tensor | None = None, *, eps: float = 1e-5, weight_offset: float = 0.0,
                   quant: int | None = None, out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                   residual_out: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                   rstd: torch.Tensor | None = None, stream=None) -> LayerNorm:
    """h = x + residual; out = (h - mean(h)) / sqrt(var(h) + eps) * (weight + weight_offset) + bias, row by row.

    Arguments as in :func:`tile_rmsnorm`.  ``bias``: N elements of weight's type (only
    with a weight).  ``mean``, ``rstd``: fp32[M] for :func:`tile_layernorm_backward`.
    New small results share a storage (see the module)."""
    if quant not in _QUANT:
        raise ValueError("quant must be None, 0, 32, 64 or 128")
    return LayerNorm(*_call("layernorm", stream, x, weight, bias, residual, eps, weight_offset, _QUANT[quant], out,
                            scales, residual_out, mean, rstd))


def tile_layernorm_backward(dy: torch.Tensor, h: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                            weight: torch.Tensor | None = None, *, dresidual: torch.Tensor | None = None,
                            weight_offset: float = 0.0, bias: bool = True, dx: torch.Tensor | None = None,
                            dweight: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                            stream=None) -> tuple[torch.Tensor, torch.Tensor | None, torch.Tensor | None]:
    """Gradient of :func:`tile_layernorm` at ``h`` (its ``residual``, or x without one):
    ``(dx, dweight, dbias)``, dx in h's type and the gradient of x and residual alike,
    dweight and dbias fp32[N] (None without a weight, dbias also with ``bias`` false,
    unless one to write is given).  ``dresidual`` and ``dx`` as in
    :func:`tile_rmsnorm_backward`.  New small results share a storage (see the module)."""
    return _call("layernorm_backward", stream, dy, h, mean, rstd, weight, dresidual, weight_offset, bias, dx, dweight,
                 dbias)


def tile_w4_matvec(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor,
                   zeros: torch.Tensor | None = None, *, group: int = 128,
                   x_scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """out[t, n] = sum_k x[t, k] (q[n, k] - zeros[n, k // group]) scales[n, k // group].

    ``x``: T x K, fp16, bf16, or e4m3 with ``x_scales`` (T x 1, or T x ceil(K /
    128)).  ``q``: uint8, N x K / 2, even columns in the low halves.  ``scales``:
    N x ceil(K / group) of fp16, bf16 or fp32; ``zeros``: uint8 of that shape
    (None: 8).  ``out``: T x N of ``out_dtype`` (default: x's type; bf16 for
    e4m3)."""
    if out_dtype is not None and out_dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported out_dtype {out_dtype}")
    return _call("w4_matvec", stream, x, q, scales, zeros, group, x_scales, out,
                 -1 if out_dtype is None else DTYPE_CODE[out_dtype])


class Mx4(NamedTuple):
    """A matrix in microscaled 4-bit floats (see include/mbtile.h for the formats).

    ``q``: uint8, M x K / 2, two e2m1 codes a byte, even columns in the low halves.
    ``scales``: uint8, one for each ``block`` columns of a row, in tiles of 128 rows
    by four blocks (ceil(M / 128) x ceil(K / block / 4) x 512): e4m3 with blocks of
    16, exponents of two plus 127 with blocks of 32.  ``tensor_scale``: with blocks of
    16, an fp32 device scalar that multiplies every value (None: 1)."""
    q: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor | None = None
    block: int = 16


def tile_mx4_quantize(x: torch.Tensor, *, block: int = 16, tensor_scale: torch.Tensor | None = None,
                      q: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None) -> Mx4:
    """``x`` (M x K, fp16, bf16 or fp32, K a multiple of 32) in 4-bit floats: a block's
    scale from its largest magnitude, each element rounded to the nearest code.

    ``tensor_scale``: with blocks of 16, what the scales are relative to; the largest
    magnitude of x divided by 448 * 6 uses their whole range.  ``q``, ``scales``:
    tensors to write.  The result holds ``tensor_scale`` itself, not a copy; new small
    codes and scales share a storage (see the module)."""
    if block not in (16, 32):
        raise ValueError("block must be 16 or 32")
    q, scales = _call("mx4_quantize", stream, x, tensor_scale, block, q, scales)
    return Mx4(q, scales, tensor_scale, block)


def _mx4(m, name: str) -> Mx4:
    if not isinstance(m, Mx4) or m.block not in (16, 32):
        raise ValueError(f"{name} must be an Mx4 with blocks of 16 or 32")
    return m


def _out_code(out, dtype, default) -> int:
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype not in DTYPE_CODE or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must be an fp16, bf16 or fp32 tensor, of the type asked for")
        return DTYPE_CODE[out.dtype]
    dtype = default if dtype is None else dtype
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported output type {dtype}")
    return DTYPE_CODE[dtype]


def tile_mx4_dequantize(m: Mx4, *, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """The values that ``m`` stands for, M x K of ``dtype`` (fp16, bf16 or fp32; default bf16)."""
    m = _mx4(m, "m")
    return _call("mx4_dequantize", stream, m.q, m.scales, m.tensor_scale, m.block, out,
                 _out_code(out, dtype, torch.bfloat16))


def tile_mx4_matmul(a: Mx4, b: Mx4, *, out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                    stream=None) -> torch.Tensor:
    """out[m, n] = sum_k a[m, k] b[n, k], summed in fp32: M x N of ``out_dtype`` (fp16,
    bf16 or fp32; default bf16) from an M x K and an N x K matrix with blocks of one size."""
    a, b = _mx4(a, "a"), _mx4(b, "b")
    if a.block != b.block:
        raise ValueError("a and b must have blocks of one size")
    return _call("mx4_matmul", stream, a.q, a.scales, a.tensor_scale, b.q, b.scales, b.tensor_scale, a.block, out,
                 _out_code(out, out_dtype, torch.bfloat16))


class _AdamwTensor(ctypes.Structure):
    """Mirror of ``mbt_adamw_tensor`` in include/mbtile.h."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("param", "grad", "exp_avg", "exp_avg_sq",
                                                     "master", "m_scales", "v_scales")]
    _fields_.append(("n", ctypes.c_int64))


class AdamwTensors:
    """The tensors that :func:`tile_adamw` updates, checked once; it holds them.
    Their data stay where they are: replace one's (``p.data = ...``) and make the
    object anew.

    ``params``: fp32, fp16 or bf16, all of one type.  ``exp_avg``, ``exp_avg_sq``:
    fp32, or e4m3 with fp32 ``m_scales`` and ``v_scales`` of ceil(n / 256)
    elements (zeros are a valid first state).  ``master``: fp32 weights beside
    16-bit params."""

    def __init__(self, params, exp_avg, exp_avg_sq, *, master=None, m_scales=None, v_scales=None):
        self.params = list(params)
        count = len(self.params)
        self._kept = {"exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq, "master": master,
                      "m_scales": m_scales, "v_scales": v_scales}
        self._kept = {k: None if v is None else list(v) for k, v in self._kept.items()}
        for name, tensors in self._kept.items():
            if tensors is not None and len(tensors) != count:
                raise ValueError(f"{name} must have one tensor per parameter")
        self.dtype = self.params[0].dtype if count else torch.float32
        self.device = self.params[0].device if count else torch.device("cuda", 0)
        self.state_dtype = self._kept["exp_avg"][0].dtype if count else torch.float32
        if self.dtype not in DTYPE_CODE or self.device.type != "cuda":
            raise ValueError("params must be fp16, bf16 or fp32 CUDA tensors")
        if self.state_dtype not in (torch.float32, E4M3):
            raise ValueError("exp_avg must be fp32 or e4m3")
        eight = self.state_dtype == E4M3
        if eight != (m_scales is not None) or eight != (v_scales is not None):
            raise ValueError("m_scales and v_scales go with e4m3 states")
        if master is not None and self.dtype == torch.float32:
            raise ValueError("master weights go with 16-bit params")
        self._rows = (_AdamwTensor * max(1, count))()
        sizes = []
        types = {"exp_avg": (self.state_dtype,), "exp_avg_sq": (self.state_dtype,), "master": _F32,
                 "m_scales": _F32, "v_scales": _F32}
        for k, p in enumerate(self.params):
            row, n = self._rows[k], p.numel()
            row.n = n
            row.param = _dense(p, f"params[{k}]", p.shape, (self.dtype,), self.device)
            for name, tensors in self._kept.items():
                if tensors is None:
                    continue
                t = tensors[k]
                want = (-(-n // ADAMW_BLOCK),) if name.endswith("scales") else t.shape
                setattr(row, name, _dense(t, f"{name}[{k}]", want, types[name], self.device))
                if not name.endswith("scales") and t.numel() != n:
                    raise ValueError(f"{name}[{k}] must have {n} elements")
            sizes.append(n)
        # the tensors that a step writes, and where their data are: replaced data (t.data = ...) are refused
        self._written = (*self.params, *(t for tensors in self._kept.values() if tensors for t in tensors))
        self._addresses = (ctypes.c_void_p * max(1, len(self._written)))(*(t.data_ptr() for t in self._written))
        self.sizes = tuple(sizes)
        self._address = ctypes.addressof(self._rows)


def tile_adamw(tensors: AdamwTensors, grads, *, step: int, lr: float, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
               grad_scale: torch.Tensor | None = None, seed: int = 0, stream=None) -> None:
    """One AdamW step in place over every tensor of ``tensors`` (see
    include/mbtile.h for the formulas and the 8-bit states' rounding).

    ``grads``: a contiguous CUDA tensor per parameter, all of one type.
    ``grad_scale``: optional fp32 device scalar that multiplies the gradients.
    ``seed``: of the 8-bit states' rounding; another one each step."""
    _call("adamw", stream, tensors._address, tensors.sizes, tensors.device.index or 0, DTYPE_CODE[tensors.dtype],
          _CODE[tensors.state_dtype], grads, step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed,
          tensors._written, ctypes.addressof(tensors._addresses))


class GradNorm(NamedTuple):
    """Results of :func:`tile_grad_norm` and :func:`tile_clip_grads`, fp32 device scalars."""
    norm: torch.Tensor
    scale: torch.Tensor


def tile_grad_norm(grads, *, max_norm: float | None = None, eps: float = 1e-6, grad_scale: torch.Tensor | None = None,
                   norm: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None) -> GradNorm:
    """norm = |grad_scale| sqrt(sum of all squares); scale = grad_scale min(1, max_norm / (norm + eps)).

    ``grads``: dense CUDA tensors on one device, fp16, bf16 and fp32 in any mixture.
    ``grad_scale``: optional fp32 device scalar that the gradients are yet to be
    multiplied by (None: 1).  ``scale`` is the factor for :func:`tile_adamw`'s
    ``grad_scale``; without ``max_norm`` it is this call's ``grad_scale``.  A new norm
    and scale share a storage (see the module)."""
    return GradNorm(*_call("grad_norm", stream, grads, grad_scale, float("inf") if max_norm is None else max_norm, eps,
                           norm, scale, False))


def tile_clip_grads(grads, max_norm: float, *, eps: float = 1e-6, grad_scale: torch.Tensor | None = None,
                    norm: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None) -> GradNorm:
    """:func:`tile_grad_norm`, and every gradient multiplied by ``scale`` in place.  No
    two of the tensors may overlap, nor one of them ``norm`` or ``scale``."""
    return GradNorm(*_call("grad_norm", stream, grads, grad_scale, max_norm, eps, norm, scale, True))

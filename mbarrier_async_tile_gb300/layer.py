"""Python binding of the layer operators: RMS norm and its gradient, the 4-bit
matrix-vector product, the AdamW step (see include/mbtile.h).

Argument marshalling and checks only, as in the package itself; results that the
caller does not provide are allocated on the stream that writes them.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import DTYPE_CODE, _check, _load

E4M3 = torch.float8_e4m3fn
MBT_E4M3 = 3
ADAMW_BLOCK = 256
_CODE = {**DTYPE_CODE, E4M3: MBT_E4M3}
_QUANT = {None: -1, 0: 0, 32: 32, 64: 64, 128: 128}


class _Functions:
    """The C functions with their argument types, looked up once."""

    def __init__(self):
        lib = _load()
        vp, i64, i32, f32, f64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                  ctypes.c_double)
        lib.tile_rmsnorm.argtypes = [vp] * 7 + [i64] * 6 + [i32] * 3 + [f32, f32, vp]
        lib.tile_rmsnorm_backward.argtypes = [vp] * 7 + [i64] * 6 + [i32] * 2 + [f32, vp]
        lib.tile_w4_matvec.argtypes = [vp] * 6 + [i64] * 6 + [i32] * 5 + [vp]
        lib.tile_adamw.argtypes = [vp, i64, i32, i32, i32, i64] + [f64] * 5 + [vp, ctypes.c_uint32, vp]
        for name in ("tile_rmsnorm", "tile_rmsnorm_backward", "tile_w4_matvec", "tile_adamw"):
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            setattr(self, name, fn)


_functions = None


def _fn() -> _Functions:
    global _functions
    if _functions is None:
        _functions = _Functions()
    return _functions


# (the current device and stream as torch's own generated code asks for them: the
# public calls build objects that cost more than a small kernel's launch)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _stream(stream, device: torch.device) -> int:
    """Handle of `stream`, or of the current stream; the tensors' device must be current."""
    index = device.index
    if index != _current_device():
        raise ValueError(f"tensors are on {device}, the current device is cuda:{_current_device()}")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device: torch.device) -> int:
    """Row pitch of a matrix that must have this shape, type and device."""
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    M, N = shape
    if M == 0 or N == 0:
        return N
    ld, step = t.stride()
    if step != 1 and N > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if M == 1:
        return N
    if ld < N:
        raise ValueError(f"{name}'s rows overlap")
    return ld


def _dense(t: torch.Tensor, name: str, shape, dtypes, device: torch.device) -> int:
    """Address of a dense tensor that must have this shape and one of the types."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)} and type "
                         f"{' or '.join(str(d) for d in dtypes)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}")
    return t.data_ptr()


def _input(t: torch.Tensor, name: str, dtypes) -> None:
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.device.type != "cuda":
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has unsupported dtype {t.dtype}")


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
    _input(x, "x", DTYPE_CODE)
    shape, dtype, device = x.shape, x.dtype, x.device
    M, N = shape
    if quant not in _QUANT:
        raise ValueError("quant must be None, 0, 32, 64 or 128")
    handle = _stream(stream, device)
    ld_x = _rows(x, "x", shape, dtype, device)
    ld_res = ld_ro = res_p = ro_p = w_p = s_p = w_code = 0
    if weight is not None:
        w_p = _dense(weight, "weight", (N,), DTYPE_CODE, device)
        w_code = DTYPE_CODE[weight.dtype]
    if residual is not None:
        ld_res = _rows(residual, "residual", shape, dtype, device)
        res_p = residual.data_ptr()
        if residual_out is None:
            residual_out = _empty(shape, dtype, device, stream)
        else:
            ld_ro = _rows(residual_out, "residual_out", shape, dtype, device)
        ro_p = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    out_dtype = dtype if quant is None else E4M3
    ld_out = 0
    if out is None:
        out = _empty(shape, out_dtype, device, stream)
    else:
        ld_out = _rows(out, "out", shape, out_dtype, device)
    if quant is not None:
        groups = -(-N // quant) if quant else 1
        if scales is None:
            scales = _empty((M, groups), torch.float32, device, stream)
            s_p = scales.data_ptr()
        else:
            s_p = _dense(scales, "scales", (M, groups), _F32, device)
    elif scales is not None:
        raise ValueError("scales need quant")
    if rstd is None:
        rstd = _empty(M, torch.float32, device, stream)
        rstd_p = rstd.data_ptr()
    else:
        rstd_p = _dense(rstd, "rstd", (M,), _F32, device)
    # (an address of 0 where a tensor is empty; the call then asks for none)
    _check(_fn().tile_rmsnorm(x.data_ptr(), res_p, w_p, out.data_ptr(), ro_p, s_p, rstd_p, M, N,
                              ld_x, ld_res, ld_out, ld_ro, DTYPE_CODE[dtype], w_code, _QUANT[quant],
                              eps, weight_offset, handle), "tile_rmsnorm")
    return RmsNorm(out, scales, residual_out, rstd)


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
    _input(h, "h", DTYPE_CODE)
    shape, dtype, device = h.shape, h.dtype, h.device
    M, N = shape
    handle = _stream(stream, device)
    ld_h = _rows(h, "h", shape, dtype, device)
    ld_dy = _rows(dy, "dy", shape, dtype, device)
    rstd_p = _dense(rstd, "rstd", (M,), _F32, device)
    w_p = w_code = res_p = ld_res = dw_p = 0
    if weight is not None:
        w_p = _dense(weight, "weight", (N,), DTYPE_CODE, device)
        w_code = DTYPE_CODE[weight.dtype]
        if dweight is None:
            dweight = _empty(N, torch.float32, device, stream)
            dw_p = dweight.data_ptr()
    if dweight is not None and not dw_p:
        dw_p = _dense(dweight, "dweight", (N,), _F32, device)
    if dresidual is not None:
        ld_res = _rows(dresidual, "dresidual", shape, dtype, device)
        res_p = dresidual.data_ptr()
    ld_dx = 0
    if dx is None:
        dx = _empty(shape, dtype, device, stream)
    else:
        ld_dx = _rows(dx, "dx", shape, dtype, device)
    _check(_fn().tile_rmsnorm_backward(dy.data_ptr(), h.data_ptr(), rstd_p, w_p, res_p,
                                       dx.data_ptr(), dw_p, M, N, ld_dy, ld_h, ld_res, ld_dx,
                                       DTYPE_CODE[dtype], w_code, weight_offset, handle),
           "tile_rmsnorm_backward")
    return dx, dweight


_X_TYPES = (torch.float16, torch.bfloat16, E4M3)
_U8 = (torch.uint8,)


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
    _input(x, "x", _X_TYPES)
    _input(q, "q", _U8)
    (T, K), device = x.shape, x.device
    N = q.shape[0]
    if q.shape[1] * 2 != K or group not in (32, 64, 128):
        raise ValueError("q must have K / 2 columns and group be 32, 64 or 128")
    handle = _stream(stream, device)
    ld_x = _rows(x, "x", x.shape, x.dtype, device)
    ld_q = _rows(q, "q", q.shape, torch.uint8, device)
    cells = (N, -(-K // group))
    s_p = _dense(scales, "scales", cells, DTYPE_CODE, device)
    z_p = 0 if zeros is None else _dense(zeros, "zeros", cells, _U8, device)
    xs_p = x_group = 0
    if x.dtype == E4M3:
        if x_scales is None or x_scales.dim() != 2:
            raise ValueError("e4m3 x needs x_scales, T x 1 or T x ceil(K / 128)")
        x_group = 0 if x_scales.shape[1] == 1 else 128
        xs_p = _dense(x_scales, "x_scales", (T, -(-K // 128) if x_group else 1), _F32, device)
    elif x_scales is not None:
        raise ValueError("x_scales need e4m3 x")
    if out is None:
        out_dtype = out_dtype or (torch.bfloat16 if x.dtype == E4M3 else x.dtype)
        if out_dtype not in DTYPE_CODE:
            raise ValueError(f"unsupported out_dtype {out_dtype}")
        out = _empty((T, N), out_dtype, device, stream)
        ld_out = 0
    elif out.dtype not in DTYPE_CODE or out_dtype not in (None, out.dtype):
        raise ValueError(f"out has dtype {out.dtype}")
    else:
        ld_out = _rows(out, "out", (T, N), out.dtype, device)
    _check(_fn().tile_w4_matvec(x.data_ptr(), xs_p, q.data_ptr(), s_p, z_p, out.data_ptr(), T, N, K,
                                ld_x, ld_q, ld_out, group, x_group, _CODE[x.dtype],
                                DTYPE_CODE[scales.dtype], DTYPE_CODE[out.dtype], handle),
           "tile_w4_matvec")
    return out


class _AdamwTensor(ctypes.Structure):
    """Mirror of ``mbt_adamw_tensor`` in include/mbtile.h."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("param", "grad", "exp_avg", "exp_avg_sq",
                                                     "master", "m_scales", "v_scales")]
    _fields_.append(("n", ctypes.c_int64))


_ROW_WORDS = ctypes.sizeof(_AdamwTensor) // 8


class AdamwTensors:
    """The tensors that :func:`tile_adamw` updates, checked once; it holds them.

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
        # the rows' grad fields, one every _ROW_WORDS words
        self._grad_pointers = (ctypes.c_uint64 * (max(1, count) * _ROW_WORDS - 1)).from_buffer(
            self._rows, _AdamwTensor.grad.offset)
        self.sizes = []
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
            self.sizes.append(n)


def tile_adamw(tensors: AdamwTensors, grads, *, step: int, lr: float, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
               grad_scale: torch.Tensor | None = None, seed: int = 0, stream=None) -> None:
    """One AdamW step in place over every tensor of ``tensors`` (see
    include/mbtile.h for the formulas and the 8-bit states' rounding).

    ``grads``: a contiguous CUDA tensor per parameter, all of one type.
    ``grad_scale``: optional fp32 device scalar that multiplies the gradients.
    ``seed``: of the 8-bit states' rounding; another one each step."""
    count = len(tensors.sizes)
    if len(grads) != count:
        raise ValueError("grads must have one tensor per parameter")
    device, rows = tensors.device, tensors._rows
    dtype = grads[0].dtype if count else torch.float32
    if dtype not in DTYPE_CODE:
        raise ValueError(f"grads have unsupported dtype {dtype}")
    handle = _stream(stream, device)
    index, pointers, at = device.index, tensors._grad_pointers, 0
    for g, n in zip(grads, tensors.sizes):
        if g.dtype is not dtype or g.numel() != n or g.get_device() != index or not g.is_contiguous():
            raise ValueError(f"grads[{at // _ROW_WORDS}] must be a contiguous {dtype} tensor of {n} elements on {device}")
        pointers[at] = g.data_ptr()
        at += _ROW_WORDS
    gs_p = 0
    if grad_scale is not None:
        gs_p = _dense(grad_scale, "grad_scale", grad_scale.shape, _F32, device)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must hold one element")
    _check(_fn().tile_adamw(rows, count, DTYPE_CODE[tensors.dtype], DTYPE_CODE[dtype],
                            _CODE[tensors.state_dtype], step, lr, beta1, beta2, eps, weight_decay,
                            gs_p, seed & 0xFFFFFFFF, handle), "tile_adamw")

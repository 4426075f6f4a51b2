"""The gradients' norm without a GPU: refusals and the descriptor's layout."""
import ctypes
import subprocess

import pytest
import torch

import mbarrier_async_tile_gb300 as mbt
from conftest import ROOT
from mbarrier_async_tile_gb300 import _build

A, B = 0x10000, 0x20000   # never dereferenced
INF = float("inf")


class Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


@pytest.fixture(scope="module", autouse=True)
def built_library():
    _build.build()


def norm(row=None, count=1, gs=0, most=1.0, eps=1e-6, to=B, scale=0):
    t = Grad(**{"grad": A, "n": 10, "dtype": 1, **(row or {})})
    return mbt.C.tile_grad_norm(ctypes.byref(t), count, gs, most, eps, to, scale, None)


@pytest.mark.parametrize("bad,code", [
    (dict(row=dict(grad=0)), -1), (dict(row=dict(n=-1)), -1), (dict(row=dict(n=1 << 41)), -1), (dict(row=dict(dtype=3)), -1),
    (dict(count=-1), -1), (dict(most=-1.0), -1), (dict(most=float("nan")), -1), (dict(eps=-1.0), -1), (dict(to=0), -1),
    (dict(row=dict(grad=A + 1)), -2), (dict(gs=A + 2), -2), (dict(to=B + 1), -2), (dict(scale=B + 2), -2),
])
def test_norm_argument_errors(bad, code):
    assert norm(**bad) == code


def scale(rows, to=B):
    t = (Grad * len(rows))(*(Grad(grad=p, n=n, dtype=d) for p, n, d in rows))
    return mbt.C.tile_grad_scale(t, len(rows), to, None)


def test_scale_argument_errors():
    assert scale([(0, 10, 1)]) == -1 and scale([(A, 10, 7)]) == -1 and scale([(A + 1, 10, 1)]) == -2
    assert scale([(A, 10, 1)], 0) == -1 and scale([(A, 10, 1)], B + 2) == -2
    # overlapping tensors, in any order and type; the same one twice
    assert scale([(A, 10, 1), (A, 10, 1)]) == -1
    assert scale([(A + 18, 10, 1), (A, 10, 1)]) == -1
    assert scale([(A, 10, 2), (A + 100, 4, 1), (A + 38, 5, 0)]) == -1
    assert mbt.C.tile_grad_scale(None, 0, None, None) == 0


def test_clip_argument_errors():
    t = (Grad * 2)(Grad(A, 10, 1, 0), Grad(A + 10, 10, 1, 0))

    def clip(count=2, gs=0, most=1.0, eps=1e-6, norm=B, to=B + 4):
        return mbt.C.tile_grad_clip(t, count, gs, most, eps, norm, to, None)

    assert clip() == -1 and clip(count=1, to=0) == -1 and clip(count=1, most=-1.0) == -1 and clip(count=1, norm=B + 2) == -2


def test_scalars_within_gradients_are_refused():
    # (a factor that one of the tensors holds would change while others are multiplied by it)
    assert scale([(A, 10, 2)], A + 36) == -1 and scale([(A, 10, 2), (B, 3, 1)], B + 4) == -1
    t = Grad(A, 10, 2, 0)

    def clip(norm, to):
        return mbt.C.tile_grad_clip(ctypes.byref(t), 1, 0, 1.0, 1e-6, norm, to, None)

    assert clip(A, B) == -1 and clip(B, A + 36) == -1 and clip(B, B) == -1


def test_python_refusals():
    for grads in ([torch.zeros(3)], [torch.zeros(3, dtype=torch.int32)], torch.zeros(2, 3), [None]):
        with pytest.raises(ValueError):
            mbt.tile_grad_norm(grads)
    with pytest.raises(TypeError):
        mbt.tile_clip_grads(None, 1.0)


def test_descriptor_matches_the_c_struct(tmp_path):
    src = tmp_path / "s.c"
    fields = [f for f, _ in Grad._fields_]
    prints = "".join(f'printf("%zu\\n", offsetof(mbt_grad, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mbtile.h"\n'
                   f'int main(void) {{ printf("%zu\\n", sizeof(mbt_grad)); {prints} return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c11", "-I", f"{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(Grad)] + [getattr(Grad, f).offset for f in fields]

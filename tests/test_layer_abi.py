"""The layer operators' argument errors, which need no GPU, and the descriptor's layout."""
import ctypes
import subprocess

import pytest

import mbarrier_async_tile_gb300 as mbt
from conftest import ROOT
from mbarrier_async_tile_gb300 import _build
from mbarrier_async_tile_gb300 import layer

A, B, C_, D = 0x10000, 0x20000, 0x30000, 0x40000   # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_library():
    _build.build()


def norm(x=A, res=0, w=B, out=C_, ro=0, scales=0, rstd=D, M=4, N=64, ld=(0, 0, 0, 0), dt=0, wdt=0, quant=-1, eps=1e-6):
    return mbt.C.tile_rmsnorm(x, res, w, out, ro, scales, rstd, M, N, *ld, dt, wdt, quant, eps, 0.0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=0), -1), (dict(out=0), -1), (dict(rstd=0), -1), (dict(M=-1), -1), (dict(N=-1), -1), (dict(dt=3), -1),
    (dict(wdt=3), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(quant=16), -3), (dict(quant=0), -1),
    (dict(scales=A), -1), (dict(ro=A), -1), (dict(ld=(63, 0, 0, 0)), -1), (dict(ld=(0, 0, 1, 0)), -1),
    (dict(x=A + 1), -2), (dict(rstd=D + 2), -2), (dict(w=B + 1), -2), (dict(M=1 << 40, N=1 << 30), -1),
])
def test_norm_argument_errors(bad, code):
    assert norm(**bad) == code


def test_norm_of_no_rows():
    assert norm(M=0, x=0, out=0, rstd=0) == 0


def grad(dy=A, h=B, rstd=C_, w=D, dres=0, dx=A, dw=D, M=4, N=64, ld=(0, 0, 0, 0), dt=1, wdt=1):
    return mbt.C.tile_rmsnorm_backward(dy, h, rstd, w, dres, dx, dw, M, N, *ld, dt, wdt, 0.0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dy=0), -1), (dict(h=0), -1), (dict(rstd=0), -1), (dict(dx=0), -1), (dict(M=-1), -1), (dict(dt=3), -1),
    (dict(ld=(0, 5, 0, 0)), -1), (dict(dx=A + 1), -2), (dict(dw=D + 2), -2), (dict(rstd=C_ + 1), -2),
])
def test_norm_gradient_argument_errors(bad, code):
    assert grad(**bad) == code
    assert grad(N=0) == 0


def w4(x=A, xs=0, q=B, s=C_, z=0, out=D, T=1, N=64, K=128, ld=(0, 0, 0), group=128, xg=0, dt=1, sdt=1, odt=1):
    return mbt.C.tile_w4_matvec(x, xs, q, s, z, out, T, N, K, *ld, group, xg, dt, sdt, odt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=0), -1), (dict(q=0), -1), (dict(s=0), -1), (dict(out=0), -1), (dict(T=-1), -1), (dict(dt=2), -1),
    (dict(sdt=3), -1), (dict(odt=3), -1), (dict(K=48), -3), (dict(group=16), -3), (dict(dt=3), -1), (dict(xs=A), -1),
    (dict(dt=3, xs=A, xg=64), -3), (dict(ld=(64, 0, 0)), -1), (dict(ld=(0, 72, 0)), -2), (dict(q=B + 8), -2),
    (dict(x=A + 1), -2), (dict(out=D + 1), -2), (dict(xg=128), -1),
])
def test_w4_argument_errors(bad, code):
    assert w4(**bad) == code
    assert w4(T=0) == 0 and w4(N=0) == 0


def adamw(row=None, count=1, pdt=2, gdt=2, sdt=2, step=1, lr=1e-3, gs=0, **kw):
    t = layer._AdamwTensor(param=A, grad=B, exp_avg=C_, exp_avg_sq=D, n=10)
    for k, v in (row or {}).items():
        setattr(t, k, v)
    return mbt.C.tile_adamw(ctypes.byref(t), count, pdt, gdt, sdt, step, lr, kw.get("b1", 0.9), 0.999, 1e-8, 0.0,
                                  gs, 0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(row=dict(param=0)), -1), (dict(row=dict(grad=0)), -1), (dict(row=dict(n=-1)), -1), (dict(count=-1), -1),
    (dict(pdt=3), -1), (dict(sdt=1), -1), (dict(step=0), -1), (dict(lr=float("nan")), -1), (dict(b1=1.0), -1),
    (dict(sdt=3), -1), (dict(row=dict(m_scales=A)), -1), (dict(row=dict(master=A)), -1),
    (dict(row=dict(param=A + 2)), -2), (dict(row=dict(exp_avg=A + 1)), -2), (dict(gs=A + 2), -2),
])
def test_adamw_argument_errors(bad, code):
    assert adamw(**bad) == code
    assert adamw(row=dict(n=0)) == 0 and adamw(count=0) == 0


def test_descriptor_matches_the_c_struct(tmp_path):
    src = tmp_path / "s.c"
    fields = [f for f, _ in layer._AdamwTensor._fields_]
    prints = "".join(f'printf("%zu\\n", offsetof(mbt_adamw_tensor, {f}));' for f in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mbtile.h"\n'
                   f'int main(void) {{ printf("%zu %d %d\\n", sizeof(mbt_adamw_tensor), MBT_ADAMW_BLOCK, MBT_E4M3); {prints} return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c11", "-I", f"{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(layer._AdamwTensor), layer.ADAMW_BLOCK, layer.MBT_E4M3] + [
        getattr(layer._AdamwTensor, f).offset for f in fields]

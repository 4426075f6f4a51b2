"""Build of libmbtile.so (the CUDA kernels and the C ABI) for sm_103a, and of
_mbtile_torch.so, the compiled half of the layer operators' Python binding.

Both are built in-tree, next to this file: each translation unit is compiled in
parallel (nvcc, and g++ for the binding), then libmbtile.so is linked with the
static CUDA runtime and the binding against it and torch's libraries.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libmbtile.so")
SOURCES = ["mbtile_kernels.cu", "mbtile_host.cpp", "mbtile_noalloc.cu", "mbtile_hostio.cpp",
           "mbtile_probe.cu", "mbtile_norm.cu", "mbtile_norm_f16.cu", "mbtile_norm_bf16.cu",
           "mbtile_norm_f32.cu", "mbtile_w4.cu", "mbtile_adamw.cu"]
BINDING = "mbtile_torch.cpp"
BINDING_PATH = os.path.join(PKG_DIR, "_mbtile_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, s) for s in [*SOURCES, BINDING]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    files.append(os.path.join(INCLUDE, "mbtile.h"))
    return files


def _stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return True
    built = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return any(os.path.getmtime(f) > built for f in _inputs())


def _run(cmd: list[str], what: str) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def _binding_flags() -> list[str]:
    import torch
    from torch.utils import cpp_extension

    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    paths = [*cpp_extension.include_paths(), os.path.join(cuda, "include"),
             sysconfig.get_paths()["include"], INCLUDE]
    return ["-O1", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(a for p in paths for a in ("-isystem", p))]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libmbtile.so if it is missing or older than its sources."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            print(res.stdout + res.stderr)
        return obj

    binding_obj = os.path.join(BUILD_DIR, "mbtile_torch.o")
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(lambda: _run(["g++", *_binding_flags(), "-c", os.path.join(CSRC, BINDING),
                                          "-o", binding_obj], f"g++ on {BINDING}"))
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "link of libmbtile.so")
    os.replace(tmp, LIB_PATH)
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, binding_obj, "-L", PKG_DIR, "-l:libmbtile.so", "-L", libs, "-ltorch_python",
          "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"],
         "link of the binding")
    os.replace(tmp, BINDING_PATH)
    return LIB_PATH

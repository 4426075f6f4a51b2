"""Build of libmbtile.so (the CUDA kernels and the C ABI) for sm_103a, and of
_mbtile_torch.so, the compiled half of the layer operators' Python binding.

Both are built in-tree, next to this file: each translation unit is compiled in
parallel (nvcc, and g++ for the binding), then libmbtile.so is linked with the
static CUDA runtime and the binding against it and torch's libraries.  The library
needs nothing of torch or Python: it is built where the binding cannot be, whose
error is then a warning here and raised by require_binding() and the calls that
need it.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sysconfig
import warnings

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
BINDING_STAMP = os.path.join(BUILD_DIR, "binding.stamp")   # which torch the binding was built for
binding_error: str | None = None   # why this process could not build it
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cuda, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _newer(path: str, sources: list[str]) -> bool:
    """Whether `path` is there and newer than the headers and these sources."""
    if not os.path.exists(path):
        return False
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")) or f in sources]
    files.append(os.path.join(INCLUDE, "mbtile.h"))
    built = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= built for f in files)


def _torch_identity() -> str:
    import torch

    return f"{torch.__version__} {os.path.dirname(torch.__file__)}"


def _binding_is_current() -> bool:
    if not _newer(BINDING_PATH, [BINDING]) or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP, encoding="utf-8") as f:
        return f.read() == _torch_identity()


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


def _compile_binding() -> str:
    obj = os.path.join(BUILD_DIR, "mbtile_torch.o")
    _run(["g++", *_binding_flags(), "-c", os.path.join(CSRC, BINDING), "-o", obj], f"g++ on {BINDING}")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG_DIR, "-l:libmbtile.so", "-L", libs, "-ltorch_python",
          "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"],
         "link of the binding")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w", encoding="utf-8") as f:
        f.write(_torch_identity())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libmbtile.so if it is missing or older than its sources, and the
    binding likewise or if it was built for another torch."""
    global binding_error
    library = force or not _newer(LIB_PATH, SOURCES)
    binding = force or (binding_error is None and not _binding_is_current())
    if not library and not binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        out = _run([nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc on {src}")
        if verbose:
            print(out)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding_obj = ex.submit(_compile_binding) if binding else None
        if library:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB_PATH + f".{os.getpid()}.tmp"
            _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "link of libmbtile.so")
            os.replace(tmp, LIB_PATH)
        if binding_obj is not None:
            try:
                _link_binding(binding_obj.result())
                binding_error = None
            except Exception as e:   # no compiler, no headers: the library stands without it
                binding_error = f"{type(e).__name__}: {e}"
                if os.path.exists(BINDING_PATH):
                    os.remove(BINDING_PATH)   # (an older one, of another library or torch)
                warnings.warn(f"the layer operators' Python binding could not be built: {binding_error[:2000]}")
    return LIB_PATH


def require_binding() -> str:
    """Path of the binding; raises if it is not there, with the reason where this process knows it."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"the layer operators' binding is not built ({BINDING_PATH}): " +
                           (binding_error or "run __graft_entry__.build() or mbarrier_async_tile_gb300._build.build()"))
    return BINDING_PATH

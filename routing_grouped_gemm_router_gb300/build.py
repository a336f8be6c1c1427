"""Build step of the C-ABI library: nvcc for sm_103a, one object per .cu, linked in-tree; then the
CPython extensions that call its training operators on torch tensors (host compiler only).

``python -m routing_grouped_gemm_router_gb300.build`` (or ``build()``) writes
``libmoe_gb300.so``, ``_native.so`` and ``_native_stack.so`` next to this file. Objects go to ``_build/`` in the package
directory. Sources are compiled in parallel; up-to-date libraries are not rebuilt. Without a
PyTorch that has CUDA libraries the extensions are left out: the C ABI does not need them.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(CSRC, "binding.cpp")
NATIVE = os.path.join(PKG, "_native.so")
NATIVE_FOR = os.path.join(OBJ, "native_for.txt")
# the second extension: source, library, what it was compiled for
STACK = (os.path.join(CSRC, "binding_stack.cpp"), os.path.join(PKG, "_native_stack.so"),
         os.path.join(OBJ, "native_stack_for.txt"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _torch_dir():
    """Where PyTorch is installed; None without one that has CUDA libraries."""
    spec = importlib.util.find_spec("torch")
    d = os.path.dirname(spec.origin) if spec and spec.origin else None
    return d if d and os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")) else None


def _native_for() -> str:
    """The Python and the PyTorch that an extension compiled now is for: it fits no other."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch_version = "of unknown version"
    return f"{sys.version} torch {torch_version} {_torch_dir()}"


def _extensions():
    return [(BINDING, NATIVE, NATIVE_FOR), STACK]


def _native_up_to_date(extension=None) -> bool:
    """Whether an extension (source, library, mark), the first by default, fits its sources and PyTorch."""
    source, native, mark = extension or _extensions()[0]
    if _torch_dir() is None:
        return True
    if not os.path.exists(mark) or open(mark).read() != _native_for():
        return False
    return os.path.exists(native) and all(
        os.path.getmtime(d) <= os.path.getmtime(native)
        for d in [source, os.path.join(CSRC, "binding.h"), __file__, *glob.glob(os.path.join(INCLUDE, "*.h"))])


def _compile_binding(source):
    """The extension's object, against the installed PyTorch's headers."""
    torch_dir, cuda = _torch_dir(), os.path.dirname(os.path.dirname(_nvcc()))
    obj = os.path.join(OBJ, os.path.basename(source) + ".o")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
           "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-c", source, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on {os.path.basename(source)}:\n{r.stderr}")
    return obj


def _link_binding(obj, native, mark):
    """An extension, next to the library that it calls."""
    tmp = native + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", tmp, obj,
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-ltorch", "-lc10_cuda", "-lc10", "-L", PKG, "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the extension failed:\n{r.stderr}")
    os.replace(tmp, native)
    with open(mark, "w") as f:
        f.write(_native_for())


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps() + [__file__])


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    """Compile every .cu under csrc/ for sm_103a and link libmoe_gb300.so, then the extensions. Returns
    the library's path."""
    os.makedirs(OBJ, exist_ok=True)
    if not force and not ptxas_info and up_to_date():
        for e in _extensions():
            if not _native_up_to_date(e):
                _link_binding(_compile_binding(e[0]), *e[1:])
        return LIB
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        bindings = [(ex.submit(_compile_binding, e[0]), e) for e in _extensions()] if _torch_dir() else []
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    for obj, (_, native, mark) in bindings:
        _link_binding(obj.result(), native, mark)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_info="--ptxas" in sys.argv))

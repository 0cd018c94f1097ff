"""Build libmla_nvfp4.so in-tree with nvcc for sm_103a (GB300), and the
Python binding of its 8-bit calls with the host compiler.

Each .cu file under csrc/ compiles to an object in parallel (binding.cpp
meanwhile), then nvcc links the shared library.  Output:
mla_attention_nvfp4_gb300/_build/libmla_nvfp4.so and _mla_fp8.torch-*.so
(git-ignored).  Either is rebuilt only when a source or header of it is newer.
The library needs neither Python nor PyTorch, and is built where the binding
cannot be.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmla_nvfp4.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def binding_name() -> str:
    """The binding is of one interpreter's and one PyTorch's ABI: its file
    name holds both, so that a tree that meets others builds another one.
    (PyTorch's version is read from its files: a C user's build imports none.)"""
    version = "none"
    spec = importlib.util.find_spec("torch")
    if spec is not None and spec.origin:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            found = re.search(r"^__version__ = ['\"]([^'\"]+)['\"]", f.read(), re.M)
        version = found.group(1) if found else "unknown"
    return f"_mla_fp8.torch-{version}{sysconfig.get_config_var('EXT_SUFFIX')}"


BINDING = os.path.join(BUILD, binding_name())


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    return "nvcc"


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "-I" + os.path.join(ROOT, "include")] + list(extra)


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "mla_nvfp4.h"), os.path.abspath(__file__)]


def _binding_deps():
    return glob.glob(os.path.join(CSRC, "*.cpp")) + [os.path.join(ROOT, "include", "mla_nvfp4.h"), os.path.abspath(__file__)]


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_up_to_date() -> bool:
    return _newer(BINDING, _binding_deps())


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


class BindingError(RuntimeError):
    """The library is built, its Python binding of the 8-bit calls is not."""


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build what is out of date.  The library needs nvcc alone: it is linked
    whatever becomes of the binding, whose failure raises BindingError after
    that."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources() if force or not library_up_to_date() else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), "-c", src, "-o", obj] + _flags(extra_flags)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding) if force or not binding_up_to_date() else None
        objs = list(ex.map(compile_one, srcs))
    if objs:
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding is not None:
        try:
            _link_binding(binding.result())
        except Exception as e:  # no compiler, no PyTorch, no headers
            raise BindingError(f"{LIB} is built; its Python binding of the 8-bit calls is not: {e}") from e
    return LIB


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile_binding() -> str:
    """binding.cpp against this interpreter's and this PyTorch's headers."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    obj = os.path.join(BUILD, "binding.o")
    _run([os.environ.get("CXX", "g++"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(root, "include"),
          "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
          "-I" + sysconfig.get_paths()["include"]])
    return obj


def _link_binding(obj: str) -> None:
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    tmp = BINDING + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
          "-ltorch", "-ltorch_cpu", "-ltorch_python", "-L" + BUILD, "-lmla_nvfp4", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    try:
        print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                    extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
    except BindingError as e:  # the C library is what this was asked for
        sys.stderr.write(f"warning: {e}\n")
        print(LIB)

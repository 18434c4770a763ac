"""Builds libgbmoe.so (the C-ABI CUDA library) in-tree for sm_103a.

Each .cu file is compiled by its own nvcc process (in parallel), then the
objects are linked into a shared library next to this file.  That takes nvcc
alone.  The C++ binding of the decode-step operators (csrc/step_bindings.cpp,
against the installed torch's headers) is compiled beside them into
_step_bindings.so, and again for another torch; without torch, which it serves,
it is left out.  Nothing is installed anywhere else.

    python -m mixture_experts_ffn_moe_gb300.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgbmoe.so")
STEPS = os.path.join(PKG, "_step_bindings.so")
STEPS_TORCH = os.path.join(BUILD, "step_bindings.torch")  # the torch that it was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgbmoe.so")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), "-c", src, "-o", obj] + NVCC_FLAGS
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _torch_version():
    """Of the installed torch; None where there is none."""
    try:
        import torch
    except ImportError:
        return None
    return str(torch.__version__)


def steps_built_against():
    """The torch version that _step_bindings.so was compiled against; None where that is not known."""
    try:
        with open(STEPS_TORCH) as f:
            return f.read()
    except OSError:
        return None


def _compile_steps(version: str) -> None:
    """The Python binding of the decode-step operators, with the host compiler."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], cuda]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE]
    for path in includes:
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "step_bindings.cpp"), "-o", STEPS + ".tmp", "-L", os.path.join(root, "lib"), "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on step_bindings.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(STEPS + ".tmp", STEPS)
    with open(STEPS_TORCH, "w") as f:
        f.write(version)


def _older(out: str, sources) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(p) > os.path.getmtime(out) for p in sources)


def _lib_stale() -> bool:
    own = [p for p in glob.glob(os.path.join(CSRC, "*")) if not p.endswith(".cpp")]
    return _older(LIB, own + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__])


def _steps_stale(version: str) -> bool:
    own = glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return _older(STEPS, own) or steps_built_against() != version


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc(), "-shared", "-o", tmp] + objs + ARCH, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgbmoe.so and _step_bindings.so if a source of theirs is newer; returns the library's path.

    The library is linked whatever becomes of the binding, whose failure is raised afterwards.
    """
    version = _torch_version()
    lib, steps = force or _lib_stale(), version is not None and (force or _steps_stale(version))
    if not lib and not steps:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_steps, version) if steps else None
        if lib:
            _link(list(ex.map(lambda s: _compile(s, verbose), srcs)))
        if binding:
            binding.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))

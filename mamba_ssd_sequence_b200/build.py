"""Builds libssd.so (the CUDA kernels and the C ABI) in-tree with nvcc for
sm_100a, and _binding.so (the compiled Python calls of the recurrence and the
norms) with g++ against torch.  Run ``python -m mamba_ssd_sequence_b200.build`` or call build().

libssd.so needs nvcc only.  Where _binding.so cannot be built (no torch, or no
headers of it), build() warns and everything but the recurrence and the norms
can be used from Python; build_binding() raises."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssd.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(OBJDIR, "_binding.txt")  # what it was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "--expt-relaxed-constexpr",
                     "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every csrc/*.cu for sm_100a and link libssd.so, and the compiled
    calls linked to it (a warning where that fails); returns the path of libssd.so."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        _try_binding()
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _try_binding(force)
    return LIB


def _try_binding(force: bool = False) -> None:
    try:
        build_binding(force)
    except Exception as e:
        if os.path.exists(BINDING):  # out of date: its calls must not be made
            os.remove(BINDING)
        warnings.warn(f"{BINDING} was not built: the recurrence and the norms cannot be called from Python ({e})")


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp into _binding.so, linked to libssd.so (which has
    to be there), unless it is newer than its sources and was built against this
    torch and Python; returns its path."""
    import sysconfig

    import torch
    built_for = f"torch {torch.__version__} {os.path.dirname(torch.__file__)} python {sys.version}"
    newest = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(INCLUDE, "ssd.h"), os.path.abspath(__file__)))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and os.path.exists(BINDING_FOR):
        with open(BINDING_FOR) as f:
            if f.read() == built_for:
                return BINDING
    from torch.utils import cpp_extension
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DSSD_TORCH_VERSION="{torch.__version__}"', "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]
    for path in cpp_extension.include_paths():
        cmd += ["-isystem", path]
    cmd += [BINDING_SRC, "-o", tmp, "-L", PKG, "-l:" + os.path.basename(LIB), "-L", torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(built_for)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_binding())

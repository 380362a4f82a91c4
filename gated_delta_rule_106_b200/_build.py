"""Build libgdn.so (all CUDA sources in csrc/) for sm_100a with nvcc, and the
Python extension ``_paged.so`` (csrc/paged_binding.cpp) with the host compiler.

Objects go to ``_build/`` at the repository root; the shared libraries are written
next to this file so that they are loaded in-tree. ``python -m
gated_delta_rule_106_b200._build`` rebuilds what is stale.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BINDING = os.path.join(PKG, "_paged.so")
BINDING_STAMP = os.path.join(OBJDIR, "_paged.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra, verbose):
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    if not _stale(obj, [src] + _headers() + [__file__]):
        return obj
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _built_for():
    """The torch and the Python whose C and C++ interfaces the extension uses."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _binding_command():
    """The compiler's arguments for the extension, its output left out."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DGDN_BUILT_FOR="{torch.__version__}"',
            "-I", INCLUDE, "-I", os.path.join(base, "include"),
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
            os.path.join(CSRC, "paged_binding.cpp"), "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]


def _build_binding(verbose):
    stamp, made = BINDING_STAMP, _built_for()
    src = os.path.join(CSRC, "paged_binding.cpp")
    if not _stale(BINDING, [src, os.path.join(INCLUDE, "gdn.h"), __file__]):
        if os.path.exists(stamp) and open(stamp).read() == made:
            return
    tmp = BINDING + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(_binding_command() + ["-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    except Exception:
        for old in (BINDING, stamp):          # of another torch, or of other sources
            if os.path.exists(old):
                os.remove(old)
        raise
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(made)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every csrc/*.cu for sm_100a and link libgdn.so, build the Python
    extension; return the library's path. Only the paged-cache calls need the extension:
    where it cannot be built (no Python or torch headers, say) that is a warning, and
    those calls raise."""
    os.makedirs(OBJDIR, exist_ok=True)
    if force:
        for f in glob.glob(os.path.join(OBJDIR, "*.o")) + glob.glob(BINDING):
            os.remove(f)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose or ptxas_info), srcs))
        refused = binding.exception()
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if refused is not None:
        warnings.warn(f"{BINDING} was not built, the paged-cache calls will raise: {refused}",
                      RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_info="--ptxas-info" in sys.argv))

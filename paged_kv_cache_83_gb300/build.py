"""Build ``_build/libpagedattn.so`` from ``csrc/*.cu`` with nvcc for sm_103a.

Each translation unit is compiled in parallel, then the objects are linked into one shared
library that exports the C ABI of ``include/pa.h``. The runtime is linked shared, so a process
that already loaded PyTorch's CUDA runtime uses that one instance. The binding's argument checks
(``csrc/args.cpp``) become an extension module for the installed PyTorch and Python. That needs a C++
compiler and the headers of both; where they are missing the library is built all the same, with a warning,
and the calls that go through the module (rotation, chunk attention, sampling) raise.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
BUILD = PKG / "_build"
LIB = BUILD / "libpagedattn.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FAST_MATH = ["--use_fast_math"]
# Subnormal logits have an order, which flushing them to zero would lose.
EXACT_MATH = {"sample.cu"}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found")


def cuda_home() -> Path:
    return Path(nvcc()).resolve().parent.parent


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _stale(out: Path, deps: list[Path]) -> bool:
    if not out.exists():
        return True
    t = out.stat().st_mtime
    return any(d.stat().st_mtime > t for d in deps)


def args_path() -> Path:
    """The extension module of csrc/args.cpp; a name of its own for each PyTorch and Python."""
    import torch
    return BUILD / f"pa_args-{torch.__version__}-{sys.implementation.cache_tag}.so"


def _build_args(headers: list[Path], force: bool) -> str:
    """Compiles csrc/args.cpp; what stood in the way, or nothing. A module of other sources does not stay then."""
    src = CSRC / "args.cpp"
    try:
        import torch
        out = args_path()
        if not (force or _stale(out, [src] + headers)):
            return ""
        home = Path(torch.__file__).resolve().parent
        tmp = out.with_suffix(f".{os.getpid()}.tmp")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-isystem{home / 'include'}",
               f"-isystem{home / 'include' / 'torch' / 'csrc' / 'api' / 'include'}",
               f"-isystem{sysconfig.get_paths()['include']}", f"-isystem{cuda_home() / 'include'}", str(src), "-o", str(tmp),
               f"-L{home / 'lib'}", "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{home / 'lib'}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
    except ImportError as e:  # no PyTorch: then no binding either
        return str(e)
    except OSError as e:  # no compiler
        lacking = str(e)
    else:
        if r.returncode == 0:
            os.replace(tmp, out)
            return ""
        lacking = f"{cmd[0]} failed on {src.name}:\n{r.stderr}"
    out.unlink(missing_ok=True)
    return lacking


def build(verbose: bool = False, force: bool = False) -> Path:
    BUILD.mkdir(parents=True, exist_ok=True)
    headers = list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh")) + [ROOT / "include" / "pa.h"]
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    f"-I{ROOT / 'include'}"]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        if force or _stale(obj, [src] + headers):
            math = [] if src.name in EXACT_MATH else FAST_MATH
            cmd = [nvcc(), *flags, *math, "-c", str(src), "-o", str(obj)]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stderr}")
            if verbose and r.stderr:
                (BUILD / (src.stem + ".ptxas.txt")).write_text(r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        args = ex.submit(_build_args, headers, force)
        objs = list(ex.map(compile_one, srcs))
        lacking = args.result()
    if force or _stale(LIB, objs):
        tmp = LIB.with_suffix(f".{os.getpid()}.tmp")
        libdir = cuda_home() / "lib64"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", *map(str, objs), "-o", str(tmp),
               "-Xlinker", f"-rpath,{libdir}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if lacking:
        warnings.warn(f"the binding's calls for rotation, chunk attention and sampling were not built: {lacking}", RuntimeWarning,
                      stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))

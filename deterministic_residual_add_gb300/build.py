"""Build libdradd.so in-tree with nvcc for sm_103a, and _binding.so, the
compiled part of the Python binding, with the host compiler.

Each .cu translation unit is compiled in parallel, then linked into a shared
library next to this file.  `python -m deterministic_residual_add_gb300.build`
builds both from the command line.

The library needs nothing but nvcc and its host compiler.  The binding, which
only the calls of train.py use, needs g++, Python's headers and a torch with
CUDA; where one of them is missing it is left out with a warning, and those
calls say so.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import threading
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = PKG / "libdradd.so"
BINDING = PKG / "_binding.so"
BINDING_SRC = CSRC / "dradd_binding.cpp"
BINDING_FOR = "binding_for.txt"  # in BUILD: the Python and torch that _binding.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No fast math: IEEE division and square root, no flush to zero, and no
# contraction of a multiply and an add into one fused operation.
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-fmad=false",
              "-prec-div=true", "-prec-sqrt=true", "-ftz=false", "-Xptxas", "-v"]

_lock = threading.Lock()


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdradd")


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _deps():
    return _sources() + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + sorted(INCLUDE.glob("*.h"))


def lib_stale() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    return any(p.stat().st_mtime > t for p in _deps())


def binding_stale() -> bool:
    """Missing, older than its sources, or built for another Python or torch
    (whose interfaces a compiled module is bound to)."""
    if not BINDING.exists():
        return True
    t = BINDING.stat().st_mtime
    if any(p.stat().st_mtime > t for p in [BINDING_SRC, *INCLUDE.glob("*.h")]):
        return True
    tag = BUILD / BINDING_FOR
    return not tag.exists() or tag.read_text() != _binding_for()


def stale() -> bool:
    return lib_stale() or (binding_stale() and not binding_lacks())


def _binding_for() -> str:
    try:
        import torch
    except ImportError:
        return f"{sys.version}\nno torch"
    return f"{sys.version}\ntorch {torch.__version__} at {Path(torch.__file__).parent}"


def binding_lacks() -> str:
    """What the binding needs and this machine does not have, or ""."""
    if not shutil.which("g++"):
        return "g++"
    if not (Path(sysconfig.get_paths()["include"]) / "Python.h").exists():
        return "Python's headers"
    try:
        import torch
    except ImportError:
        return "torch"
    root = Path(torch.__file__).resolve().parent
    if not (root / "include/c10/cuda/CUDAStream.h").exists() or not (root / "lib/libc10_cuda.so").exists():
        return "a torch with CUDA"
    return ""


def _binding_flags():
    """Compiler flags against the installed torch and Python."""
    import torch

    root = Path(torch.__file__).resolve().parent
    inc = [root / "include", root / "include/torch/csrc/api/include", Path(nvcc()).resolve().parents[1] / "include",
           Path(sysconfig.get_paths()["include"]), INCLUDE]
    return ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in inc)], root / "lib"


def _run(cmd, what: str):
    r = subprocess.run([str(c) for c in cmd], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _build_lib(ex: ThreadPoolExecutor):
    cc = nvcc()

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-I", str(INCLUDE), "-I", str(CSRC), "-c", str(src),
               "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        (BUILD / (src.stem + ".ptxas.txt")).write_text(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src.name}:\n{r.stdout}\n{r.stderr}")
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB.with_suffix(f".so.tmp{os.getpid()}")
    _run([cc, *ARCH, "-shared", "-o", tmp, *objs], "linking the library")
    os.replace(tmp, LIB)


def _compile_binding() -> Path:
    flags, _ = _binding_flags()
    obj = BUILD / "dradd_binding.o"
    _run(["g++", *flags, "-c", BINDING_SRC, "-o", obj], "compiling the binding")
    return obj


def _link_binding(obj: Path):
    """Against libdradd.so beside it; torch's libraries are loaded already
    when the module is imported."""
    _, libs = _binding_flags()
    tmp = BINDING.with_suffix(f".so.tmp{os.getpid()}")
    _run(["g++", "-shared", obj, "-o", tmp, f"-L{LIB.parent}", "-ldradd", "-Wl,-rpath,$ORIGIN", f"-L{libs}", "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], "linking the binding")
    os.replace(tmp, BINDING)
    (BUILD / BINDING_FOR).write_text(_binding_for())


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile and link what is missing or older than its sources: libdradd.so,
    then _binding.so."""
    with _lock:
        BUILD.mkdir(exist_ok=True)
        lacks = binding_lacks()
        want_lib = force or lib_stale()
        want_binding = not lacks and (force or binding_stale())
        with ThreadPoolExecutor(len(_sources()) + 1) as ex:
            binding = ex.submit(_compile_binding) if want_binding else None
            if want_lib:
                _build_lib(ex)
                if verbose:
                    for f in sorted(BUILD.glob("*.ptxas.txt")):
                        print(f.read_text())
            if binding:
                _link_binding(binding.result())
        if lacks and binding_stale():
            warnings.warn(f"{LIB.name} is built; {BINDING.name} is not, for want of {lacks}: dropout, the gradients and "
                          "the rotary calls will not load", stacklevel=2)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

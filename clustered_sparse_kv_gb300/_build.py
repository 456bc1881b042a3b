"""Build step of the CUDA library: nvcc, sm_103a only, objects compiled in parallel.

Produces ``libwaveindex.so`` and the extension module ``_paged.so`` (the paged cache's argument checks, host C++
against this Python's torch) inside the package directory (in-tree, git-ignored).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libwaveindex.so")
EXT = os.path.join(PKG, "_paged.so")
STAMP = os.path.join(BUILD, "paged_binding.stamp")  # what EXT was built against

SOURCES = ["wi_api.cu", "wi_build.cu", "wi_decode.cu", "wi_dense.cu", "wi_assign_tc.cu", "wi_noalloc.cu",
           "wi_grow.cu", "wi_tier.cu", "wi_selftest.cu", "wi_paged_api.cu", "wi_paged.cu", "wi_paged_attn.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def _torch_of_this_python() -> str:
    """The Python and the torch that the extension module reads the insides of."""
    import importlib.metadata
    import importlib.util
    import sys

    spec = importlib.util.find_spec("torch")
    return f"{sys.version} | torch {importlib.metadata.version('torch')} in {spec.origin if spec else None}\n"


def is_current() -> bool:
    """Whether both files are there, newer than their sources, and the extension module fits this Python and torch."""
    if not all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime() for f in (LIB, EXT)):
        return False
    try:
        with open(STAMP) as f:
            return f.read() == _torch_of_this_python()
    except OSError:
        return False


def _run(what: str, cmd: list[str]):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_ext() -> str:
    import sysconfig

    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "paged_binding.o")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    _run("g++ for paged_binding.cpp", ["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{d}" for d in dirs], "-c",
                                       os.path.join(CSRC, "paged_binding.cpp"), "-o", obj])
    return obj


def _link_ext(obj: str):
    from torch.utils import cpp_extension

    dirs = cpp_extension.library_paths()
    tmp = EXT + f".tmp{os.getpid()}"
    _run("link of _paged.so", ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libwaveindex.so", "-Wl,-rpath,$ORIGIN",
                               *[f"-L{d}" for d in dirs], *[f"-Wl,-rpath,{d}" for d in dirs], "-ltorch_python",
                               "-ltorch_cpu", "-lc10"])
    os.replace(tmp, EXT)
    with open(STAMP, "w") as f:
        f.write(_torch_of_this_python())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and is_current():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_ext(ext.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))

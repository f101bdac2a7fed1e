"""Build of the sm_103a CUDA library ``libck_gb300.so`` (in-tree, no cmake).

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel for
``-gencode arch=compute_103a,code=sm_103a`` only, then linked into one shared
library under ``swiglu_mlp_group_gb300/_build/``.  nvcc cross-compiles, so the
build also runs on machines without a GPU.

``csrc/torch_calls.cpp``, the Python binding's quick calls, is compiled by g++
beside it where torch's and Python's headers are there, for that torch; without
it the same calls go through ctypes.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libck_gb300.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")


def calls_path() -> str | None:
    """Where the quick calls for the installed torch belong; None without torch."""
    try:
        return os.path.join(BUILD_DIR, f"ck_torch_calls-{importlib.metadata.version('torch')}.so")
    except importlib.metadata.PackageNotFoundError:
        return None


def _calls_dirs() -> tuple[str, str, str] | None:
    """(torch's folder, Python's headers, CUDA's headers), or None if one of them is missing."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None or calls_path() is None or shutil.which("g++") is None:
        return None
    try:
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    except RuntimeError:
        return None
    dirs = (os.path.dirname(spec.origin), sysconfig.get_paths()["include"], os.path.join(cuda, "include"))
    heads = (os.path.join(dirs[0], "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(dirs[1], "Python.h"), os.path.join(dirs[2], "cuda_runtime_api.h"))
    return dirs if all(os.path.exists(h) for h in heads) else None


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libck_gb300.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + [CALLS_SOURCE] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    built = [LIB_PATH] + ([calls_path()] if _calls_dirs() else [])
    if not all(os.path.exists(b) for b in built):
        return False
    t = min(os.path.getmtime(b) for b in built)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link the library; returns its path.  Raises on any failure."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    dirs = _calls_dirs()
    calls_obj = os.path.join(BUILD_DIR, "torch_calls.o")

    def compile_calls() -> None:
        torch_dir, python_inc, cuda_inc = dirs
        includes = [INCLUDE, os.path.join(torch_dir, "include"),
                    os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), python_inc, cuda_inc]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", CALLS_SOURCE, "-o", calls_obj]
        r = subprocess.run(cmd + [f"-I{i}" for i in includes], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}")

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        calls = ex.submit(compile_calls) if dirs else None
        objs = list(ex.map(compile_one, srcs))
        if calls:
            calls.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcuda"] * 0
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if dirs:
        tmp = calls_path() + f".tmp{os.getpid()}"
        cmd = ["g++", "-shared", "-o", tmp, calls_obj, "-L", BUILD_DIR, f"-l:{LIB_NAME}", "-L", os.path.join(dirs[0], "lib"),
               "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-ltorch_cuda", "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, calls_path())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))

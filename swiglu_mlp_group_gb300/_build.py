"""Build of the sm_103a CUDA library ``libck_gb300.so`` (in-tree, no cmake).

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel for
``-gencode arch=compute_103a,code=sm_103a`` only, then linked into one shared
library under ``swiglu_mlp_group_gb300/_build/``.  nvcc cross-compiles, so the
build also runs on machines without a GPU.

``csrc/torch_calls.cpp``, the Python binding's quick calls, is compiled by g++
beside it where torch's and Python's headers are there, for that torch and that
Python.  It uses what torch keeps to itself, which another torch may have
otherwise: where it does not compile or link, the build warns and goes on, and
the same calls go through ctypes.
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
import warnings

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
    """Where the quick calls for the installed torch and this Python belong; None without torch."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None
    return os.path.join(BUILD_DIR, f"ck_torch_calls-{version}{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def _calls_failed() -> str:
    """The file that says why the quick calls could not be built."""
    return calls_path() + ".failed"


def _remove(path: str) -> None:
    if os.path.exists(path):
        os.remove(path)


def _calls_dirs() -> tuple[str, str, str] | None:
    """(torch's folder, Python's headers, CUDA's headers), or None if one of them or torch's CUDA part is missing."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None or calls_path() is None or shutil.which("g++") is None:
        return None
    try:
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    except RuntimeError:
        return None
    dirs = (os.path.dirname(spec.origin), sysconfig.get_paths()["include"], os.path.join(cuda, "include"))
    heads = (os.path.join(dirs[0], "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(dirs[0], "lib", "libc10_cuda.so"),
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
    built = [LIB_PATH]
    if _calls_dirs():
        built.append(calls_path() if os.path.exists(calls_path()) else _calls_failed())
    if not all(os.path.exists(b) for b in built):
        return False
    t = min(os.path.getmtime(b) for b in built)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile_calls(dirs: tuple[str, str, str], obj: str) -> str | None:
    """Compile the quick calls; the compiler's messages if it fails."""
    torch_dir, python_inc, cuda_inc = dirs
    includes = [INCLUDE, os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), python_inc, cuda_inc]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", CALLS_SOURCE, "-o", obj]
    r = subprocess.run(cmd + [f"-I{i}" for i in includes], capture_output=True, text=True)
    return None if r.returncode == 0 else f"g++ failed for {CALLS_SOURCE}:\n{r.stdout}\n{r.stderr}"


def _link_calls(dirs: tuple[str, str, str], obj: str) -> str | None:
    """Link the quick calls against the library; the linker's messages if it fails."""
    tmp = calls_path() + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.dirname(LIB_PATH), f"-l:{LIB_NAME}", "-L",
           os.path.join(dirs[0], "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-ltorch_cuda",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return f"link failed:\n{r.stdout}\n{r.stderr}"
    os.replace(tmp, calls_path())
    return None


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link the library; returns its path.  Raises on any failure but one of the quick calls."""
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

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        calls = ex.submit(_compile_calls, dirs, calls_obj) if dirs else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcuda"] * 0
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if calls:
        why = calls.result() or _link_calls(dirs, calls_obj)
        if why:
            with open(_calls_failed(), "w") as f:
                f.write(why)
            warnings.warn(f"the compiled calls were not built, and go through ctypes: {why}", RuntimeWarning, stacklevel=2)
    if calls_path() and (not calls or why):  # one of an older library
        _remove(calls_path())
    elif calls:
        _remove(_calls_failed())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))

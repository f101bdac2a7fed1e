"""The compiled calls' own checks (csrc/torch_calls.cpp) on the host: the source is compiled with host tensors and a
library that records and fills (torch_calls_check.cc).  What they hand to the library has to be what the Python calls
would hand it; anything else they have to leave to Python (None, and no call)."""
import ctypes
import os
import subprocess
from importlib.machinery import ExtensionFileLoader
from importlib.util import module_from_spec, spec_from_file_location

import pytest
import torch

from swiglu_mlp_group_gb300 import _build

BF16 = torch.bfloat16
T, H = 9, 64


class Check:
    def __init__(self, path):
        spec = spec_from_file_location("ck_torch_calls", path, loader=ExtensionFileLoader("ck_torch_calls", path))
        self.quick = module_from_spec(spec)
        spec.loader.exec_module(self.quick)
        self.so = ctypes.CDLL(path)
        self.so.check_ldm.restype = ctypes.c_int64

    def taken(self, name, *args):
        """Whether the call reached the library."""
        before = self.so.check_calls()
        got = getattr(self.quick, name)(*args)
        made = self.so.check_calls() - before
        assert made == (0 if got is None else 1)
        return got is not None


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    dirs = _build._calls_dirs()
    if dirs is None:
        pytest.skip("torch's, Python's or CUDA's headers are not there")
    torch_dir, python_inc, cuda_inc = dirs
    path = str(tmp_path_factory.mktemp("calls") / "ck_torch_calls.so")
    here = os.path.dirname(os.path.abspath(__file__))
    includes = [_build.INCLUDE, _build.CSRC, os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), python_inc, cuda_inc]
    cmd = ["g++", "-O0", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", os.path.join(here, "torch_calls_check.cc"),
           "-o", path] + [f"-I{i}" for i in includes]
    cmd += ["-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return Check(path)


def rows(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def norm_args(x, branch, gate=None, scale=None, shift=None, per=0, fp4=False, **out):
    if fp4:
        return ("block_norm_fp4", x, branch, "nv", 1.0, None, gate, 1.0, 1.0, "rms", None, None, scale, shift, per, 1e-6,
                out.get("h_out"), out.get("codes"), out.get("scales"))
    return ("block_norm", x, branch, None, gate, 1.0, 1.0, "rms", None, None, scale, shift, per, 1e-6, out.get("h_out"),
            out.get("n_out"))


@pytest.mark.parametrize("fp4", [False, True])
def test_modulation_rows(check, fp4):
    """Several groups: rows of gate, scale and shift lie at one stride of at least H.  One row for all samples
    (`v.expand(groups, H)`, stride 0) is no such stride: the row behind the first one is not its memory."""
    x, b = rows(T, H), rows(T, H)
    mod = rows(3, 3 * H)
    gate, scale, shift = mod[:, :H], mod[:, H:2 * H], mod[:, 2 * H:]
    one = mod[:1, :H].expand(3, H)
    assert check.taken(*norm_args(x, b, gate, scale, shift, 4, fp4)) and check.so.check_ldm() == 3 * H
    assert check.taken(*norm_args(x, b, None, None, shift.contiguous(), 4, fp4)) and check.so.check_ldm() == H
    for mods in ((one, None, None), (None, one, None), (None, None, one), (one, one, one), (one, scale, None), (scale, one, None),
                 (one, None, shift.contiguous()), (None, shift.contiguous(), one), (gate, scale, shift.contiguous())):
        assert not check.taken(*norm_args(x, b, *mods, 4, fp4)), [None if m is None else m.stride() for m in mods]
    short = mod.as_strided((3, H), (H // 2, 1))
    assert not check.taken(*norm_args(x, b, short, None, None, 4, fp4))
    # one group reads one row, wherever the others are
    for per in (0, T, 100):
        assert check.taken(*norm_args(x, b, one, scale, short, per, fp4)) and check.so.check_ldm() == H
    assert check.taken(*norm_args(rows(4, H), rows(4, H), one, one, one, 4, fp4))


MARK = 0x5a
U8 = torch.uint8


def bytes_of(t):
    return t.contiguous().view(U8)


def test_outputs_that_share_their_memory(check):
    """An output that still shares its memory with the tensor it was lazily cloned from gets its own before it is
    written: the other tensor keeps its values, and the call's are in the output."""
    N = 32
    x, b = rows(T, H), rows(T, H)
    w, ws = rows(N, H // 2, dtype=U8), rows(512, dtype=U8)
    codes, scales = rows(T, H // 2, dtype=U8), rows(512, dtype=U8)
    gu, gus = rows(4 * H, H // 2, dtype=U8), rows(2 * 512, dtype=U8)
    d, ds = rows(H, H, dtype=U8), rows(2 * 512, dtype=U8)
    y, h, n, c, s = rows(T, N), rows(T, H), rows(T, H), codes.clone(), scales.clone()
    for given, call in [
        ((y,), lambda y: ("fp4_gemm", codes, scales, w, ws, "nv", 1.0, None, None, y)),
        ((y,), lambda y: ("fp4_gemm", codes, scales, w, ws, "nv", 1.0, None, y, y)),
        ((y,), lambda y: ("fp4_linear", x, w, ws, "nv", 1.0, 1.0, None, "none", y, None, None)),
        ((h,), lambda h: ("fp4_swiglu_mlp", h, gu, gus, d, ds, "nv", 1.0, 1.0, 1.0, 1.0, None, None, h, h, None)),
        ((c, s), lambda c, s: ("fp4_quantize", x, "nv", 1.0, "none", c, s)),
        ((h, n), lambda h, n: norm_args(x, b, h_out=h, n_out=n)),
        ((h, n), lambda h, n: norm_args(h, n, h_out=h, n_out=n)),
        ((h, c, s), lambda h, c, s: norm_args(x, b, fp4=True, h_out=h, codes=c, scales=s)),
    ]:
        kept = [t.clone() for t in given]
        clones = [torch._lazy_clone(t) for t in given]
        args = call(*clones)
        assert check.taken(*args), args[0]
        for t, k, o in zip(given, kept, clones):
            assert torch.equal(t, k), f"{args[0]}: the tensor behind an output was written"
            assert (bytes_of(o) == MARK).all(), f"{args[0]}: the output was not written"


def test_odd_columns_are_not_halved(check):
    """[gate | up] has an even number of columns; of 2K + 1 the last would be left out without a word."""
    wide = rows(T, 4 * H)
    w, ws = rows(32, H // 2, dtype=U8), rows(512, dtype=U8)
    for cols, ok in ((2 * H, True), (2 * H + 1, False)):
        x = wide[:, :cols]
        assert check.taken("fp4_quantize", x, "nv", 1.0, "swiglu", None, None) == ok
        assert check.taken("fp4_linear", x, w, ws, "nv", 1.0, 1.0, None, "swiglu", None, None, None) == ok

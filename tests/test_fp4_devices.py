"""Tensors of the 4-bit operators and of the block norm lie on one device, and that is
the current one; outputs and workspaces that a call makes lie there, too.  Checked with
stand-ins for tensors, which name their device and have no memory."""
import pytest
import torch

import swiglu_mlp_group_gb300 as ck
from test_attention_devices import Stub

U8, F32 = torch.uint8, torch.float32
M, K, N, I = 5, 64, 24, 96


class Library:
    """Every operator records its name and succeeds; sizes are as the library has them."""

    def __init__(self, calls):
        self.calls = calls

    def ck_fp4_scale_bytes(self, fmt, rows, cols):
        word = 64 if fmt == ck.CK_FP4_NV else 128
        return -(-rows // 128) * -(-cols // word) * 512

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(ck, "lib", lambda: Library(made))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return made


def tiled(rows, cols):
    return Stub((-(-rows // 128) * -(-cols // 64) * 512,), U8)


def vec(*shape, dtype=torch.bfloat16):
    return Stub(shape, dtype)


CALLS = {
    "fp4_quantize": dict(x=vec(M, K), fmt="nv", codes=vec(M, K // 2, dtype=U8), scales=tiled(M, K)),
    "fp4_gemm": dict(codes=vec(M, K // 2, dtype=U8), scales=tiled(M, K), W=vec(N, K // 2, dtype=U8), w_scales=tiled(N, K),
                     fmt="nv", bias=vec(N), residual=vec(M, N), out=vec(M, N)),
    "fp4_linear": dict(x=vec(M, K), W=vec(N, K // 2, dtype=U8), w_scales=tiled(N, K), fmt="nv", bias=vec(N),
                       residual=vec(M, N), out=vec(M, N), workspace=vec(1 << 20, dtype=U8)),
    "fp4_swiglu_mlp": dict(x=vec(M, K), Wgu=vec(2 * I, K // 2, dtype=U8), gu_scales=tiled(2 * I, K),
                           Wd=vec(K, I // 2, dtype=U8), d_scales=tiled(K, I), fmt="nv", bgu=vec(2 * I), bd=vec(K),
                           residual=vec(M, K), out=vec(M, K), workspace=vec(1 << 20, dtype=U8)),
    "block_norm": dict(x=vec(M, K), branch=vec(M, K), post_weight=vec(K, dtype=F32), gate=vec(3, K), scale=vec(3, K),
                       shift=vec(3, K), tokens_per_group=2, weight=vec(K, dtype=F32), bias=vec(K, dtype=F32),
                       h_out=vec(M, K), n_out=vec(M, K)),
    "block_norm_fp4": dict(x=vec(M, K), branch=vec(M, K), fmt="nv", weight=vec(K), h_out=vec(M, K),
                           codes=vec(M, K // 2, dtype=U8), scales=tiled(M, K)),
}
TENSORS = [(c, n) for c, a in CALLS.items() for n, v in a.items() if isinstance(v, Stub)]


def moved(a, names, dev):
    return {n: Stub(v.shape, v.dtype, dev) if n in names else v for n, v in a.items()}


@pytest.mark.parametrize("call", list(CALLS))
def test_one_device_is_accepted(call, calls):
    getattr(ck, call)(**CALLS[call])
    assert calls == ["ck_" + call]


@pytest.mark.parametrize("dev", [-1, 1])
@pytest.mark.parametrize("call,name", TENSORS)
def test_one_tensor_elsewhere(call, name, dev, calls):
    with pytest.raises(ValueError):
        getattr(ck, call)(**moved(CALLS[call], [name], dev))
    assert not calls


@pytest.mark.parametrize("call", list(CALLS))
def test_all_on_a_device_that_is_not_current(call, calls, monkeypatch):
    names = [n for n, v in CALLS[call].items() if isinstance(v, Stub)]
    with pytest.raises(ValueError):
        getattr(ck, call)(**moved(CALLS[call], names, 1))
    assert not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    getattr(ck, call)(**moved(CALLS[call], names, 1))
    assert calls == ["ck_" + call]


@pytest.mark.parametrize("call,name,shape", [("fp4_gemm", "W", (N, K)), ("fp4_gemm", "scales", (511,)), ("fp4_gemm", "bias", (N + 1,)),
                                             ("fp4_gemm", "out", (M, N + 8)), ("fp4_linear", "residual", (M + 1, N)),
                                             ("fp4_swiglu_mlp", "Wd", (K, I)), ("fp4_swiglu_mlp", "bgu", (I,)),
                                             ("block_norm", "gate", (2, K)), ("block_norm", "n_out", (M, K + 8)),
                                             ("block_norm_fp4", "codes", (M, K)), ("block_norm_fp4", "scales", (64,))])
def test_a_shape_that_does_not_fit(call, name, shape, calls):
    a = dict(CALLS[call])
    a[name] = Stub(shape, a[name].dtype)
    with pytest.raises(ValueError):
        getattr(ck, call)(**a)
    assert not calls


def test_compiled_calls_take_no_host_tensors():
    """They hand tensors of the host, stand-ins and wrong counts back to Python."""
    quick = ck._quick()
    if quick is None:
        pytest.skip("torch's headers are not there")
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    for name, n in (("fp4_quantize", 6), ("fp4_gemm", 9), ("fp4_linear", 11), ("fp4_swiglu_mlp", 15), ("block_norm", 15),
                    ("block_norm_fp4", 18)):
        call = getattr(quick, name)
        assert call() is None and call(*[None] * n) is None and call(*[x] * n) is None and call(*[vec(M, K)] * n) is None

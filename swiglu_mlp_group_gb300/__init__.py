"""GB300 (sm_103a) ConvRot INT8 W8A8 linear, fused SwiGLU MLP, small-M GEMV and the
attention between a block's qkv and output projections.

Python binding of the C ABI in ``include/ck.h`` (library ``libck_gb300.so``).
The ``ck_*`` functions below are the C entry points themselves (ctypes); the
lower-case helpers only marshal torch tensors (device memory, streams) into
those calls -- every step of the computation runs in the library's CUDA
kernels.  There is no CPU or PyTorch fallback: if the library is missing or the
device is not a GB300, the calls raise.

The method (web pages, cited by title and section): comfy-kitchen PR #277
"FP16 tensor-core fallback for int8_linear" (The key observation), sglang PR
#44196 "comfy_kitchen SwiGLU MLP for Qwen-Image 2.1" (Motivation), sglang PR
#35994 report "Load serialized Comfy ConvRot INT8 DiTs" (kitchen_int8.py
excerpt), comfy-kitchen PR #248 "Performance improvements for qwen 3.x
(Part 2)" (Description).
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings

__all__ = [
    "CkError", "lib", "library_path", "build",
    "CK_OK", "CK_ERR_NULL", "CK_ERR_SHAPE", "CK_ERR_DTYPE", "CK_ERR_GROUP", "CK_ERR_ALIGN",
    "CK_ERR_WORKSPACE", "CK_ERR_UNSUPPORTED_DEVICE", "CK_ERR_CUDA", "CK_ERR_TIMEOUT",
    "CK_ERR_INVALID", "CK_ERR_INDEX", "CK_ROPE_HALF", "CK_ROPE_INTERLEAVED", "CK_F32", "CK_BF16", "CK_ACT_NONE", "CK_ACT_SWIGLU",
    "CK_WLAYOUT_ROWMAJOR_I8", "CK_WLAYOUT_GEMM_F16", "CK_WLAYOUT_GEMV_PACKED",
    "CK_WLAYOUT_GEMV_PACKED_W6", "CK_WLAYOUT_GEMV_PACKED_W4", "CK_WLAYOUT_GEMM_F16_GLU",
    "GEMV_LAYOUT_OF_BITS",
    "CK_OP_INT8_LINEAR", "CK_OP_SWIGLU_MLP", "CK_OP_GEMV_SMALLM", "CK_OP_DEBUG_GEMM_S32",
    "quantize_weight", "rotate_quantize_act", "prepare_weight", "int8_linear", "swiglu_mlp",
    "gemv_smallM", "quantize_weight_bits", "packed_gemv_dequant", "debug_int8_gemm_s32", "poll_device_status", "set_wait_timeout_ns",
    "set_launch_overlap", "debug_stalled_wait", "workspace_bytes",
    "qk_norm_rope", "kv_append", "prefix_attention", "prefix_attention_workspace", "cross_attention",
    "cross_attention_workspace",
    "CK_FP4_MX", "CK_FP4_NV", "CK_NORM_RMS", "CK_NORM_LAYER",
    "fp4_quantize", "fp4_tile_scales", "fp4_gemm", "fp4_linear", "fp4_linear_workspace", "fp4_swiglu_mlp",
    "fp4_swiglu_mlp_workspace", "block_norm", "block_norm_fp4",
]

# ck_status
CK_OK, CK_ERR_NULL, CK_ERR_SHAPE, CK_ERR_DTYPE, CK_ERR_GROUP, CK_ERR_ALIGN = 0, 1, 2, 3, 4, 5
CK_ERR_WORKSPACE, CK_ERR_UNSUPPORTED_DEVICE, CK_ERR_CUDA, CK_ERR_TIMEOUT, CK_ERR_INVALID = (
    6, 7, 8, 9, 10)
CK_ERR_INDEX = 11
# ck_rope_mode
CK_ROPE_HALF, CK_ROPE_INTERLEAVED = 0, 1
# ck_dtype, ck_input_act, ck_wlayout, ck_op
CK_F32, CK_BF16 = 0, 1
CK_ACT_NONE, CK_ACT_SWIGLU = 0, 1
CK_WLAYOUT_ROWMAJOR_I8, CK_WLAYOUT_GEMM_F16, CK_WLAYOUT_GEMV_PACKED = 0, 1, 2
CK_WLAYOUT_GEMV_PACKED_W6, CK_WLAYOUT_GEMV_PACKED_W4, CK_WLAYOUT_GEMM_F16_GLU = 3, 4, 5
# the GEMV-resident layout of each weight code width
GEMV_LAYOUT_OF_BITS = {8: CK_WLAYOUT_GEMV_PACKED, 6: CK_WLAYOUT_GEMV_PACKED_W6,
                       4: CK_WLAYOUT_GEMV_PACKED_W4}
CK_OP_INT8_LINEAR, CK_OP_SWIGLU_MLP, CK_OP_GEMV_SMALLM, CK_OP_DEBUG_GEMM_S32 = 0, 1, 2, 3

# ck_fp4_format, ck_norm
CK_FP4_MX, CK_FP4_NV = 0, 1
CK_NORM_RMS, CK_NORM_LAYER = 0, 1

_ROPES = {"half": CK_ROPE_HALF, "interleaved": CK_ROPE_INTERLEAVED}
_ACTS = {"none": CK_ACT_NONE, "swiglu": CK_ACT_SWIGLU}
_FP4S = {"mx": CK_FP4_MX, "nv": CK_FP4_NV}
_NORMS = {"rms": CK_NORM_RMS, "layer": CK_NORM_LAYER}

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None

_i64, _vp, _sz, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_f32 = ctypes.c_float
# name -> (restype, argtypes), in the order of include/ck.h
_SIGNATURES = {
    "ck_status_string": (ctypes.c_char_p, [_int]),
    "ck_version": (_int, []),
    "ck_device_check": (_int, []),
    "ck_convrot_quantize_weight": (_int, [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp]),
    "ck_convrot_quantize_weight_bits": (_int, [_vp, _int, _i64, _i64, _int, _int, _vp, _vp, _vp]),
    "ck_rotate_quantize_act": (_int, [_vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp]),
    "ck_rotate_quantize_act_f16": (_int, [_vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp]),
    "ck_int8_gemm_dequant": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp]),
    "ck_prepared_weight_bytes": (_sz, [_int, _i64, _i64]),
    "ck_prepare_weight": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]),
    "ck_workspace_bytes": (_sz, [_int, _i64, _i64, _i64, _int]),
    "ck_int8_linear": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _int, _vp, _i64, _int, _vp, _vp,
                              _vp, _vp, _sz, _vp]),
    "ck_int8_linear_noalloc": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _vp, _i64, _int, _vp, _vp,
                                      _vp, _vp]),
    "ck_swiglu_mlp": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int,
                             _vp, _vp, _sz, _vp]),
    "ck_int8_gemv_smallM": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _i64, _int, _vp, _vp, _vp,
                                   _vp, _sz, _vp]),
    "ck_int8_gemv_dequant": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "ck_packed_gemv_smallM": (_int, [_vp, _i64, _i64, _i64, _int, _vp, _int, _i64, _int, _vp, _vp,
                                     _vp, _vp, _sz, _vp]),
    "ck_packed_gemv_dequant": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _i64, _vp, _vp, _vp, _vp]),
    "ck_qk_norm_rope": (_int, [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _int, _i64, _i64, _f32, _vp,
                               _i64, _i64, _int, _vp, _vp, _i64, _vp, _i64, _vp]),
    "ck_kv_append": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _int, _f32, _vp, _i64, _i64,
                            _int, _vp, _vp, _vp, _vp, _i64, _i64, _vp]),
    "ck_prefix_attention": (_int, [_vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp,
                                   _i64, _vp, _i64, _vp, _i64, _f32, _vp, _i64, _vp, _sz, _vp]),
    "ck_prefix_attention_workspace_bytes": (_sz, [_i64] * 7),
    "ck_cross_attention": (_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64,
                                  _vp, _f32, _vp, _i64, _vp, _sz, _vp]),
    "ck_cross_attention_workspace_bytes": (_sz, [_i64] * 6),
    "ck_fp4_scale_bytes": (_sz, [_int, _i64, _i64]),
    "ck_fp4_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _int, _int, _f32, _vp, _vp, _vp]),
    "ck_fp4_tile_scales": (_int, [_vp, _i64, _i64, _int, _vp, _vp]),
    "ck_fp4_gemm": (_int, [_vp, _vp, _i64, _i64, _int, _vp, _vp, _i64, _f32, _vp, _vp, _vp, _vp]),
    "ck_fp4_linear": (_int, [_vp, _i64, _i64, _i64, _int, _int, _f32, _vp, _vp, _f32, _i64, _vp, _vp, _vp,
                             _vp, _sz, _vp]),
    "ck_fp4_linear_workspace_bytes": (_sz, [_i64, _i64, _int]),
    "ck_fp4_swiglu_mlp": (_int, [_vp, _i64, _i64, _i64, _int, _f32, _vp, _vp, _f32, _vp, _f32, _vp, _vp,
                                 _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "ck_fp4_swiglu_mlp_workspace_bytes": (_sz, [_i64, _i64, _i64, _int]),
    "ck_block_norm": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _f32,
                             _int, _vp, _vp, _int, _f32, _vp, _i64, _vp, _i64, _vp]),
    "ck_block_norm_fp4": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _f32,
                                 _f32, _int, _vp, _vp, _int, _f32, _vp, _i64, _int, _f32, _vp, _vp, _vp]),
    "ck_poll_device_status": (_int, [_vp]),
    "ck_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "ck_set_launch_overlap": (None, [_int]),
    "ck_debug_int8_gemm_s32": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]),
    "ck_measure_int8_mma_tops": (_int, [ctypes.POINTER(ctypes.c_double), _vp, _vp]),
    "ck_measure_tcgen05_f16_tflops": (_int, [ctypes.POINTER(ctypes.c_double), _vp]),
    "ck_debug_gemv_s32": (_int, [_vp, _i64, _i64, _vp, _int, _i64, _vp, _vp]),
    "ck_debug_force_gemm_tile": (None, [_int]),
    "ck_debug_gemm_tile_choice": (_int, [_i64, _i64, _i64, _int]),
    "ck_debug_force_gemv_quantizer": (None, [_int]),
    "ck_debug_stalled_wait": (_int, [_vp]),
}


class CkError(RuntimeError):
    """A ck_* call returned a status other than CK_OK."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_string(status)}")


def library_path() -> str:
    from . import _build
    return _build.LIB_PATH


def build(force: bool = False) -> str:
    """Compile libck_gb300.so for sm_103a (nvcc); returns its path."""
    from . import _build
    return _build.build(force=force)


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


_quick_module = False  # not looked for yet


def _quick():
    """The compiled calls (csrc/torch_calls.cpp) of the 4-bit operators and the block norm, or None where they were
    not built or do not load.  Such a call returns None where anything is not in order, and the Python one says what."""
    global _quick_module
    if _quick_module is False:
        from importlib.machinery import ExtensionFileLoader
        from importlib.util import module_from_spec, spec_from_file_location

        from . import _build
        _torch()
        lib()
        path, module = _build.calls_path(), None
        if path is not None and os.path.exists(path):
            spec = spec_from_file_location("ck_torch_calls", path, loader=ExtensionFileLoader("ck_torch_calls", path))
            try:
                module = module_from_spec(spec)
                spec.loader.exec_module(module)
            except ImportError as e:  # of another build of torch
                module = None
                warnings.warn(f"the compiled calls do not load, and go through ctypes: {e}", RuntimeWarning, stacklevel=3)
        _quick_module = module
    return _quick_module


def _make_entry(name):
    def entry(*args):
        return getattr(lib(), name)(*args)
    entry.__name__ = name
    entry.__doc__ = f"The C entry point {name} of include/ck.h (ctypes)."
    return entry


for _name in _SIGNATURES:
    globals()[_name] = _make_entry(_name)
    __all__.append(_name)


def status_string(st: int) -> str:
    return lib().ck_status_string(int(st)).decode()


def _check(st: int, where: str) -> None:
    if st != CK_OK:
        raise CkError(st, where)


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _check_residual(residual, M: int, N: int) -> None:
    """A residual must be a contiguous bf16 [M, N] tensor (the library reads rows of N)."""
    if residual is None:
        return
    torch = _torch()
    if residual.dtype != torch.bfloat16 or tuple(residual.shape) != (M, N) or \
            not residual.is_contiguous():
        raise ValueError(f"residual must be a contiguous bf16 tensor of shape ({M}, {N})")


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("expected contiguous CUDA tensors")


def workspace_bytes(op: int, M: int, K: int, N: int, wlayout: int = CK_WLAYOUT_GEMM_F16) -> int:
    return int(lib().ck_workspace_bytes(op, M, K, N, wlayout))


def _workspace(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def quantize_weight(W, g: int, stream=None):
    """Offline ConvRot weight quantization -> (Wq int8 [N, K], sw f32 [N])."""
    torch = _torch()
    _require_cuda(W)
    N, K = W.shape
    wdt = {torch.float32: CK_F32, torch.bfloat16: CK_BF16}[W.dtype]
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sw = torch.empty((N,), dtype=torch.float32, device=W.device)
    _check(lib().ck_convrot_quantize_weight(W.data_ptr(), wdt, N, K, g, Wq.data_ptr(),
                                            sw.data_ptr(), _stream(stream)),
           "ck_convrot_quantize_weight")
    return Wq, sw


def quantize_weight_bits(W, g: int, bits: int, stream=None):
    """ConvRot weight quantization to b-bit codes (bits 8, 6 or 4: W8A8 / W6A8 /
    W4A8) -> (Wq int8 [N, K] within +-(2^(bits-1) - 1), sw f32 [N])."""
    torch = _torch()
    _require_cuda(W)
    N, K = W.shape
    wdt = {torch.float32: CK_F32, torch.bfloat16: CK_BF16}[W.dtype]
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sw = torch.empty((N,), dtype=torch.float32, device=W.device)
    _check(lib().ck_convrot_quantize_weight_bits(W.data_ptr(), wdt, N, K, g, int(bits), Wq.data_ptr(),
                                                 sw.data_ptr(), _stream(stream)),
           "ck_convrot_quantize_weight_bits")
    return Wq, sw


def rotate_quantize_act(x, g: int, act: str = "none", K: int | None = None, stream=None):
    """Online activation rotation + per-token quantization -> (xq int8 [M, K], sx f32 [M])."""
    torch = _torch()
    _require_cuda(x)
    M, ldx = x.shape
    if K is None:
        K = ldx // 2 if act == "swiglu" else ldx
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(lib().ck_rotate_quantize_act(x.data_ptr(), M, K, ldx, _ACTS[act], g, xq.data_ptr(),
                                        sx.data_ptr(), _stream(stream)), "ck_rotate_quantize_act")
    return xq, sx


def rotate_quantize_act_f16(x, g: int, act: str = "none", K: int | None = None, stream=None):
    """Activation quantization with fp16-held codes -> (xq16 fp16 [M, K], sx f32 [M])."""
    torch = _torch()
    _require_cuda(x)
    M, ldx = x.shape
    if K is None:
        K = ldx // 2 if act == "swiglu" else ldx
    xq = torch.empty((M, K), dtype=torch.float16, device=x.device)
    sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(lib().ck_rotate_quantize_act_f16(x.data_ptr(), M, K, ldx, _ACTS[act], g, xq.data_ptr(),
                                            sx.data_ptr(), _stream(stream)),
           "ck_rotate_quantize_act_f16")
    return xq, sx


def int8_gemm_dequant(xq16, sx, W16, sw, bias=None, out=None, stream=None, residual=None):
    """GEMM + dequant on fp16-held codes and a CK_WLAYOUT_GEMM_F16 weight -> y bf16 [M, N]
    (+ residual bf16 [M, N], which may be `out` itself)."""
    torch = _torch()
    _require_cuda(xq16, sx, W16, sw, bias, residual)
    M, K = xq16.shape
    N = sw.shape[0]
    _check_residual(residual, M, N)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq16.device)
    _check(lib().ck_int8_gemm_dequant(xq16.data_ptr(), sx.data_ptr(), M, K, W16.data_ptr(),
                                      sw.data_ptr(), N, _ptr(bias), _ptr(residual), y.data_ptr(),
                                      _stream(stream)),
           "ck_int8_gemm_dequant")
    return y


def measure_int8_mma_tops(stream=None) -> float:
    """Dense mma.sync s8 throughput of the current device (TOPS)."""
    torch = _torch()
    v = ctypes.c_double(0.0)
    sink = torch.zeros(4, dtype=torch.int32, device="cuda")
    _check(lib().ck_measure_int8_mma_tops(ctypes.byref(v), sink.data_ptr(), _stream(stream)),
           "ck_measure_int8_mma_tops")
    return v.value


def measure_tcgen05_f16_tflops(stream=None) -> float:
    """Issue rate of tcgen05.mma kind::f16 128x256x16 on the whole device (TFLOP/s)."""
    v = ctypes.c_double(0.0)
    _check(lib().ck_measure_tcgen05_f16_tflops(ctypes.byref(v), _stream(stream)),
           "ck_measure_tcgen05_f16_tflops")
    return v.value


def prepare_weight(Wq, sw, layout: int, stream=None):
    """Re-lay a quantized weight into a resident layout (a flat uint8 device tensor)."""
    torch = _torch()
    _require_cuda(Wq, sw)
    N, K = Wq.shape
    nbytes = int(lib().ck_prepared_weight_bytes(layout, N, K))
    if nbytes == 0:
        raise CkError(CK_ERR_SHAPE, "ck_prepared_weight_bytes")
    out = torch.empty((nbytes,), dtype=torch.uint8, device=Wq.device)
    _check(lib().ck_prepare_weight(Wq.data_ptr(), _ptr(sw), N, K, layout, out.data_ptr(), nbytes,
                                   _stream(stream)), "ck_prepare_weight")
    return out


def int8_linear(x, W, sw, g: int, bias=None, act: str = "none", N: int | None = None,
                wlayout: int = CK_WLAYOUT_ROWMAJOR_I8, out=None, workspace=None, stream=None,
                residual=None):
    """ConvRot W8A8 linear y = bf16(acc * sx * sw + bias + residual) -> y bf16 [M, N]."""
    torch = _torch()
    _require_cuda(x, W, sw, bias, residual)
    M, ldx = x.shape
    K = ldx // 2 if act == "swiglu" else ldx
    if N is None:
        N = sw.shape[0]
    _check_residual(residual, M, N)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    need = workspace_bytes(CK_OP_INT8_LINEAR, M, K, N, wlayout)
    ws = workspace if workspace is not None else _workspace(need, x.device)
    _check(lib().ck_int8_linear(x.data_ptr(), M, K, ldx, _ACTS[act], W.data_ptr(), wlayout,
                                sw.data_ptr(), N, g, _ptr(bias), _ptr(residual), y.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(stream)), "ck_int8_linear")
    return y


def swiglu_mlp(x, Wgu, sgu, Wd, sd, g: int, bgu=None, bd=None,
               wlayout: int = CK_WLAYOUT_ROWMAJOR_I8, out=None, workspace=None, stream=None,
               residual=None):
    """Fused SwiGLU MLP: packed [gate | up] linear, then the swiglu-quantized down linear
    (whose epilogue adds `residual`, bf16 [M, H], if given)."""
    torch = _torch()
    _require_cuda(x, Wgu, sgu, Wd, sd, bgu, bd, residual)
    M, H = x.shape
    I = sgu.shape[0] // 2
    _check_residual(residual, M, H)
    y = out if out is not None else torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    need = workspace_bytes(CK_OP_SWIGLU_MLP, M, H, I, wlayout)
    ws = workspace if workspace is not None else _workspace(need, x.device)
    _check(lib().ck_swiglu_mlp(x.data_ptr(), M, H, I, Wgu.data_ptr(), sgu.data_ptr(), _ptr(bgu),
                               Wd.data_ptr(), sd.data_ptr(), _ptr(bd), _ptr(residual), wlayout, g,
                               y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
           "ck_swiglu_mlp")
    return y


def gemv_smallM(x, Wpacked, N: int, g: int, bias=None, act: str = "none", out=None,
                workspace=None, stream=None, residual=None, wlayout: int = CK_WLAYOUT_GEMV_PACKED):
    """Small-M (M <= 8) GEMV over a GEMV-resident layout (INT8, or the W6A8 / W4A8
    ones) -> y bf16 [M, N] (+ residual)."""
    torch = _torch()
    _require_cuda(x, Wpacked, bias, residual)
    M, ldx = x.shape
    K = ldx // 2 if act == "swiglu" else ldx
    _check_residual(residual, M, N)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    need = workspace_bytes(CK_OP_GEMV_SMALLM, M, K, N)
    ws = workspace if workspace is not None else _workspace(need, x.device)
    if wlayout == CK_WLAYOUT_GEMV_PACKED:
        _check(lib().ck_int8_gemv_smallM(x.data_ptr(), M, K, ldx, _ACTS[act], Wpacked.data_ptr(), N,
                                         g, _ptr(bias), _ptr(residual), y.data_ptr(), ws.data_ptr(),
                                         ws.numel(), _stream(stream)), "ck_int8_gemv_smallM")
    else:
        _check(lib().ck_packed_gemv_smallM(x.data_ptr(), M, K, ldx, _ACTS[act], Wpacked.data_ptr(),
                                           wlayout, N, g, _ptr(bias), _ptr(residual), y.data_ptr(),
                                           ws.data_ptr(), ws.numel(), _stream(stream)),
               "ck_packed_gemv_smallM")
    return y


def int8_gemv_dequant(xq, sx, Wpacked, N: int, bias=None, out=None, stream=None, residual=None):
    """Small-M GEMV + dequant on INT8 codes (rotate_quantize_act) and a packed weight -> y bf16 [M, N]."""
    torch = _torch()
    _require_cuda(xq, sx, Wpacked, bias, residual)
    if xq.dtype != torch.int8:
        raise TypeError("int8_gemv_dequant takes the INT8 codes of rotate_quantize_act")
    M, K = xq.shape
    _check_residual(residual, M, N)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check(lib().ck_int8_gemv_dequant(xq.data_ptr(), sx.data_ptr(), M, K, Wpacked.data_ptr(), N,
                                      _ptr(bias), _ptr(residual), y.data_ptr(), _stream(stream)),
           "ck_int8_gemv_dequant")
    return y


def packed_gemv_dequant(xq, sx, Wpacked, wlayout: int, N: int, bias=None, out=None, stream=None,
                        residual=None):
    """int8_gemv_dequant over any GEMV-resident layout (INT8, W6A8, W4A8) -> y bf16 [M, N]."""
    torch = _torch()
    _require_cuda(xq, sx, Wpacked, bias, residual)
    if xq.dtype != torch.int8:
        raise TypeError("packed_gemv_dequant takes the INT8 codes of rotate_quantize_act")
    M, K = xq.shape
    _check_residual(residual, M, N)
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check(lib().ck_packed_gemv_dequant(xq.data_ptr(), sx.data_ptr(), M, K, Wpacked.data_ptr(),
                                        wlayout, N, _ptr(bias), _ptr(residual), y.data_ptr(),
                                        _stream(stream)), "ck_packed_gemv_dequant")
    return y


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _call_device(x, what: str) -> int:
    """Index of the device of a call: x's.  The library launches on the current one, so it has to be that."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev != _torch().cuda.current_device():
        raise ValueError(f"{what} is on cuda:{dev}, which is not the current device")
    return dev


def _token_stride(x, shape, what: str, dev: int) -> int:
    """Elements from one token of x (bf16 [..., heads, D] on the call's device, of this shape) to the next: its
    heads lie next to each other, its tokens at one stride throughout."""
    if x.dtype is not _torch().bfloat16 or x.get_device() != dev:
        raise ValueError(f"{what} must be a bf16 tensor on cuda:{dev}")
    st = x.stride()
    H, D = shape[-2], shape[-1]
    ld = H * D
    if (st[-2] != D and H > 1) or (st[-1] != 1 and D > 1):
        raise ValueError(f"{what}: the heads of a token must lie next to each other")
    if len(shape) == 4:
        B, n = shape[0], shape[1]
        if n > 1:
            ld = st[1]
            if B > 1 and st[0] != n * ld:
                raise ValueError(f"{what}: tokens must lie at one stride over batch and length")
        elif B > 1:
            ld = st[0]
    elif shape[0] > 1:
        ld = st[0]
    return ld


def _typed(t, dtype, what: str, dev: int, shape=None):
    """Data pointer of an optional contiguous tensor of the given type (and shape) on the call's device."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{what} must be a contiguous tensor of {dtype} on cuda:{dev}")


def _given_workspace(ws, dev: int):
    """A caller's workspace: any contiguous memory on the call's device."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return ws


def _run_stream(stream, dev: int) -> int:
    """The stream a call runs on: the one given, or the device's current one (its handle alone: building a
    Stream object for it takes 3 us of a small call's 10)."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _new_like(x, stream):
    """A new contiguous tensor like x (whose rows _token_stride has passed) that belongs to the call's stream."""
    torch = _torch()
    if stream is None:
        return torch.empty_like(x)  # x's tokens are contiguous or have gaps: contiguous either way
    with torch.cuda.stream(stream):
        return torch.empty_like(x)


def _new(shape, dtype, like, stream):
    """A new tensor that belongs to the stream the call runs on."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _new_on(shape, dtype, device, stream):
    """A new tensor of the call's stream (device: a torch.device, x's; an index is 2 us of a small call's 10)."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rotation(cos_sin, positions, T: int, mode: str, dev: int):
    """(table pointer, max_pos, rot_dim, mode, positions pointer) of the rotation arguments."""
    torch = _torch()
    rope = _ROPES.get(mode)
    if rope is None:
        raise ValueError("mode must be 'half' or 'interleaved'")
    if cos_sin is None:
        return None, 0, 0, rope, None
    if positions is None:
        raise ValueError("a rotation needs positions")
    max_pos, rot = cos_sin.shape
    return (_typed(cos_sin, torch.float32, "cos_sin", dev), max_pos, rot, rope,
            _typed(positions, torch.int32, "positions", dev, (T,)))


def _norm_weight(w, D: int, what: str, dtype, dev: int):
    """Data pointer of an optional norm weight [D] of the given type."""
    return None if w is None else _typed(w, dtype, what, dev, (D,))


def _weight_type(*ws):
    """(torch type, ck_dtype) of optional norm weights: f32 if the first one given is, else bf16."""
    torch = _torch()
    for w in ws:
        if w is not None:
            return (torch.float32, CK_F32) if w.dtype is torch.float32 else (torch.bfloat16, CK_BF16)
    return torch.bfloat16, CK_BF16


def qk_norm_rope(q, k, cos_sin=None, positions=None, wq=None, wk=None, eps: float = 1e-6,
                 mode: str = "half", q_out=None, k_out=None, stream=None):
    """RMS norm of each query / key head (where wq / wk is given) and the position rotation
    (where cos_sin is) in one pass -> (q_out, k_out).

    q [T, Hq, D], k [T, Hk, D] or None, bf16: views of a packed projection's rows will do.  cos_sin f32
    [max_pos, rot_dim] (cosines, then sines), positions int32 [T].  wq, wk [D], f32 or bf16 alike.
    q_out=q, k_out=k work in place."""
    shape = q.shape
    T, Hq, D = shape
    dev = _call_device(q, "q")
    ldq = _token_stride(q, shape, "q", dev)
    table, max_pos, rot, rope, pos = _rotation(cos_sin, positions, T, mode, dev)
    dt, wdt = _weight_type(wq, wk)
    if q_out is None:
        q_out, ldqo = _new_like(q, stream), Hq * D
    elif q_out.shape != shape:
        raise ValueError("q_out must have q's shape")
    else:
        ldqo = _token_stride(q_out, shape, "q_out", dev)
    if k is None:
        k_out = pk = pko = None
        Hk = ldk = ldko = 0
    else:
        kshape = k.shape
        Hk = kshape[1]
        if kshape[0] != T or kshape[2] != D:
            raise ValueError("q and k must have the same tokens and head size")
        ldk = _token_stride(k, kshape, "k", dev)
        if k_out is None:
            k_out, ldko = _new_like(k, stream), Hk * D
        elif k_out.shape != kshape:
            raise ValueError("k_out must have k's shape")
        else:
            ldko = _token_stride(k_out, kshape, "k_out", dev)
        pk, pko = k.data_ptr(), k_out.data_ptr()
    st = lib().ck_qk_norm_rope(
        q.data_ptr(), ldq, Hq, _norm_weight(wq, D, "wq", dt, dev), pk, ldk, Hk, _norm_weight(wk, D, "wk", dt, dev), wdt,
        T, D, eps, table, max_pos, rot, rope, pos, q_out.data_ptr(), ldqo, pko, ldko, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_qk_norm_rope")
    return q_out, k_out


def _caches(k_cache, v_cache, dev: int):
    """(shape, pointers) of a paged cache: contiguous bf16 [pages, Hkv, page_size, D], twice."""
    bf16 = _torch().bfloat16
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("a cache is [pages, Hkv, page_size, D]")
    return shape, _typed(k_cache, bf16, "k_cache", dev), _typed(v_cache, bf16, "v_cache", dev, shape)


def kv_append(k, v, k_cache, v_cache, slots, cos_sin=None, positions=None, wk=None, eps: float = 1e-6,
              mode: str = "half", stream=None) -> None:
    """Write T tokens' keys (normed where wk is given, rotated where cos_sin is) and values into the
    pages of a cache.

    k, v [T, Hkv, D] bf16 (views of a packed projection's rows will do); k_cache, v_cache bf16
    [pages, Hkv, page_size, D]; slots int64 [T] = page * page_size + row, negative: skip the token."""
    shape = k.shape
    T, H, D = shape
    dev = _call_device(k, "k")
    (pages, Hc, page_size, Dc), pkc, pvc = _caches(k_cache, v_cache, dev)
    if v.shape != shape or Hc != H or Dc != D:
        raise ValueError("k, v and the caches must have the same heads and head size")
    table, max_pos, rot, rope, pos = _rotation(cos_sin, positions, T, mode, dev)
    dt, wdt = _weight_type(wk)
    st = lib().ck_kv_append(
        k.data_ptr(), _token_stride(k, shape, "k", dev), v.data_ptr(), _token_stride(v, shape, "v", dev), T, H, D,
        _norm_weight(wk, D, "wk", dt, dev), wdt, eps, table, max_pos, rot, rope, pos,
        _typed(slots, _torch().int64, "slots", dev, (T,)), pkc, pvc, pages, page_size, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_kv_append")


def prefix_attention_workspace(q, k_cache, prefix_len: int, max_seq_len: int, stream=None):
    """A workspace for prefix_attention calls of these sizes (q [B, Lq, Hq, D])."""
    B, Lq, Hq, D = q.shape
    n = int(lib().ck_prefix_attention_workspace_bytes(B, Lq, Hq, k_cache.shape[1], D, prefix_len, max_seq_len))
    return _new((max(n, 16),), _torch().uint8, q, stream)


def prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len: int, block_table, seq_lens,
                     max_seq_len: int, scale: float | None = None, out=None, workspace=None, stream=None):
    """Attention of B sequences behind a shared prefix over a paged cache -> bf16 [B, Lq, Hq, D].

    q [B, Lq, Hq, D] bf16: the last Lq of each sequence's seq_lens[b] own cached tokens; token i sees the
    prefix and the own tokens 0 .. seq_lens[b] - Lq + i.  prefix_pages int32 [ceil(prefix_len / page_size)],
    block_table int32 [B, >= ceil(max_seq_len / page_size)], seq_lens int32 [B].  scale: 1 / sqrt(D) if None."""
    torch = _torch()
    shape = q.shape
    B, Lq, Hq, D = shape
    dev = _call_device(q, "q")
    (pages, H, page_size, Dc), pkc, pvc = _caches(k_cache, v_cache, dev)
    if Dc != D:
        raise ValueError("q and the caches must have the same head size")
    ldq = _token_stride(q, shape, "q", dev)
    i32 = torch.int32
    pp = _typed(prefix_pages, i32, "prefix_pages", dev)
    if prefix_len > 0 and (pp is None or prefix_pages.numel() * page_size < prefix_len):
        raise ValueError("prefix_pages must hold prefix_len tokens")
    bt, width = _typed(block_table, i32, "block_table", dev), 0
    if bt is not None:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must have a row for every sequence")
        width = block_table.shape[1]
    if out is None:
        out, ldo = _new_like(q, stream), Hq * D
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    else:
        ldo = _token_stride(out, shape, "out", dev)
    ws = (_given_workspace(workspace, dev) if workspace is not None else
          prefix_attention_workspace(q, k_cache, prefix_len, max_seq_len, stream))
    st = lib().ck_prefix_attention(
        q.data_ptr(), ldq, B, Lq, Hq, H, D, pkc, pvc, pages, page_size, pp, prefix_len, bt, width,
        _typed(seq_lens, i32, "seq_lens", dev, (B,)), max_seq_len, D ** -0.5 if scale is None else scale,
        out.data_ptr(), ldo, ws.data_ptr(), ws.nbytes, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_prefix_attention")
    return out


def cross_attention_workspace(q, k, stream=None):
    """A workspace for cross_attention calls of these sizes (q [B, Lq, Hq, D], k [B, Lk, Hkv, D])."""
    B, Lq, Hq, D = q.shape
    n = int(lib().ck_cross_attention_workspace_bytes(B, Lq, k.shape[1], Hq, k.shape[2], D))
    return _new((max(n, 16),), _torch().uint8, q, stream)


def cross_attention(q, k, v, kv_lens=None, scale: float | None = None, out=None, workspace=None, stream=None):
    """Attention of q [B, Lq, Hq, D] over states k, v [B, Lk, Hkv, D], the first kv_lens[b] (int32 [B];
    None: all) of them real -> bf16 [B, Lq, Hq, D].  scale: 1 / sqrt(D) if None."""
    torch = _torch()
    shape, kshape = q.shape, k.shape
    B, Lq, Hq, D = shape
    if v.shape != kshape or len(kshape) != 4 or kshape[0] != B or kshape[3] != D:
        raise ValueError("k and v must be [B, Lk, Hkv, D] of q's batch and head size")
    Lk, H = kshape[1], kshape[2]
    dev = _call_device(q, "q")
    ldq = _token_stride(q, shape, "q", dev)
    ldk, ldv = (_token_stride(k, kshape, "k", dev), _token_stride(v, kshape, "v", dev)) if Lk > 0 else (0, 0)
    if out is None:
        out, ldo = _new_like(q, stream), Hq * D
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    else:
        ldo = _token_stride(out, shape, "out", dev)
    ws = _given_workspace(workspace, dev) if workspace is not None else cross_attention_workspace(q, k, stream)
    st = lib().ck_cross_attention(
        q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, B, Lq, Lk, Hq, H, D,
        _typed(kv_lens, torch.int32, "kv_lens", dev, (B,)), D ** -0.5 if scale is None else scale,
        out.data_ptr(), ldo, ws.data_ptr(), ws.nbytes, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_cross_attention")
    return out


# ---------------------------------------------------------------------------
# microscaled 4-bit floats, block norms
# ---------------------------------------------------------------------------

def _row_stride(x, dtype, what: str, dev: int, shape=None) -> int:
    """Elements from one row of x (2-D, of this type and shape, on the call's device) to the next."""
    xs = x.shape
    if x.dtype is dtype and x.get_device() == dev and (xs == shape if shape is not None else len(xs) == 2):
        ld, inner = x.stride()
        if inner == 1 or xs[1] <= 1:
            return ld if xs[0] > 1 else xs[1]
        raise ValueError(f"{what}: the elements of a row must lie next to each other")
    if len(xs) != 2 or (shape is not None and xs != shape):
        raise ValueError(f"{what} must have shape {'[rows, columns]' if shape is None else tuple(shape)}")
    raise ValueError(f"{what} must be a tensor of {dtype} on cuda:{dev}")


def _fp4_format(fmt: str) -> int:
    f = _FP4S.get(fmt)
    if f is None:
        raise ValueError("fmt must be 'mx' or 'nv'")
    return f


def _act(act: str) -> int:
    a = _ACTS.get(act)
    if a is None:
        raise ValueError("act must be 'none' or 'swiglu'")
    return a


def _tokens(x, act: int):
    """(M, K) of a call's x [M, K], or of its [gate | up], 2K columns."""
    M, K = x.shape
    if act != CK_ACT_SWIGLU:
        return M, K
    if K % 2 != 0:
        raise ValueError("x must hold [gate | up], an even number of columns")
    return M, K // 2


def _tiled_bytes(f: int, rows: int, K: int) -> int:
    """ck_fp4_scale_bytes, without its refusals (a call's own come before a tensor is used)."""
    return (rows + 127) // 128 * ((K + 63) // 64 if f == CK_FP4_NV else (K + 127) // 128) * 512


def _fp4_operand(codes, scales, f: int, what: str, dev: int):
    """(rows, K, pointers) of codes [rows, K / 2] and their tiled scales."""
    u8 = _torch().uint8
    shape = codes.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be codes [rows, K / 2]")
    rows, half = shape
    p, ps = _typed(codes, u8, what, dev), _typed(scales, u8, "scales", dev)
    if scales.numel() < (rows + 127) // 128 * (half + 31 >> 5 if f else half + 63 >> 6) * 512:
        raise ValueError(f"{what}'s scales must be tiled scales of these codes")
    return rows, 2 * half, p, ps


def _out_rows(out, M: int, N: int, dev: int, device, stream):
    """A linear's output (contiguous bf16 [M, N]): the one given, checked, or a new one."""
    torch = _torch()
    if out is not None:
        _typed(out, torch.bfloat16, "out", dev, (M, N))
        return out
    return _new_on((M, N), torch.bfloat16, device, stream)


def _scales_out(scales, n: int, dev: int, device, stream):
    """Tiled scales to write: the tensor given, if it is large enough, or a new one."""
    u8 = _torch().uint8
    if scales is None:
        return _new_on((n,), u8, device, stream)
    _typed(scales, u8, "scales", dev)
    if scales.nbytes < n:
        raise ValueError(f"scales must hold {n} bytes")
    return scales


def fp4_quantize(x, fmt: str, scale: float = 1.0, act: str = "none", codes=None, scales=None, stream=None):
    """Quantize x [M, K] (bf16 or f32; act "swiglu": bf16 [gate | up] of 2K columns; rows may lie apart) to
    microscaled 4-bit floats -> (codes uint8 [M, K / 2], tiled scales uint8).

    fmt "mx": 32 codes share a power of two; "nv": 16 codes share an E4M3 number, the tensor `scale`."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.fp4_quantize(x, fmt, scale, act, codes, scales)
        if got is not None:
            return got
    torch = _torch()
    f, a = _fp4_format(fmt), _act(act)
    dev = _call_device(x, "x")
    f32 = x.dtype is torch.float32
    ldx = _row_stride(x, torch.float32 if f32 else torch.bfloat16, "x", dev)
    M, K = _tokens(x, a)
    n = int(lib().ck_fp4_scale_bytes(f, M, K))
    if n == 0:
        raise CkError(CK_ERR_SHAPE, "ck_fp4_quantize")
    if codes is None:
        codes = _new_on((M, K // 2), torch.uint8, x.device, stream)
    scales = _scales_out(scales, n, dev, x.device, stream)
    st = lib().ck_fp4_quantize(x.data_ptr(), CK_F32 if f32 else CK_BF16, M, K, ldx, a, f, scale,
                               _typed(codes, torch.uint8, "codes", dev, (M, K // 2)), scales.data_ptr(),
                               _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_fp4_quantize")
    return codes, scales


def fp4_tile_scales(scales, fmt: str, stream=None):
    """Block scales by row (a checkpoint's: uint8 [rows, K / 32] "mx", [rows, K / 16] "nv") -> tiled."""
    torch = _torch()
    f = _fp4_format(fmt)
    dev = _call_device(scales, "scales")
    p = _typed(scales, torch.uint8, "scales", dev)
    if scales.dim() != 2:
        raise ValueError("scales must be [rows, blocks]")
    rows, K = scales.shape[0], scales.shape[1] * (32 if f == CK_FP4_MX else 16)
    n = int(lib().ck_fp4_scale_bytes(f, rows, K))
    if n == 0:
        raise CkError(CK_ERR_SHAPE, "ck_fp4_tile_scales")
    out = _new_on((n,), torch.uint8, scales.device, stream)
    st = lib().ck_fp4_tile_scales(p, rows, K, f, out.data_ptr(), _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_fp4_tile_scales")
    return out


def fp4_gemm(codes, scales, W, w_scales, fmt: str, alpha: float = 1.0, bias=None, residual=None, out=None,
             stream=None):
    """y = bf16(alpha X W^T + bias + residual) -> bf16 [M, N], X of codes [M, K / 2] and W of [N, K / 2] with
    tiled scales (fp4_quantize, block_norm_fp4, fp4_tile_scales).  residual may be out."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.fp4_gemm(codes, scales, W, w_scales, fmt, alpha, bias, residual, out)
        if got is not None:
            return got
    f = _fp4_format(fmt)
    dev = _call_device(codes, "codes")
    M, K, px, pxs = _fp4_operand(codes, scales, f, "codes", dev)
    N, Kw, pw, pws = _fp4_operand(W, w_scales, f, "W", dev)
    if Kw != K:
        raise ValueError("codes and W must have the same columns")
    bf16 = _torch().bfloat16
    pb, pr = _typed(bias, bf16, "bias", dev, (N,)), _typed(residual, bf16, "residual", dev, (M, N))
    y = _out_rows(out, M, N, dev, codes.device, stream)
    st = lib().ck_fp4_gemm(px, pxs, M, K, f, pw, pws, N, alpha, pb, pr, y.data_ptr(), _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_fp4_gemm")
    return y


def fp4_linear_workspace(M: int, K: int, fmt: str, device="cuda", stream=None):
    """A workspace for fp4_linear calls of M tokens and K columns."""
    n = int(lib().ck_fp4_linear_workspace_bytes(M, K, _fp4_format(fmt)))
    return _new_on((max(n, 16),), _torch().uint8, device, stream)


def fp4_linear(x, W, w_scales, fmt: str, x_scale: float = 1.0, w_scale: float = 1.0, bias=None, act: str = "none",
               out=None, workspace=None, residual=None, stream=None):
    """Linear on 4-bit weights -> bf16 [M, N]: x [M, K] bf16 (act "swiglu": [gate | up]; rows may lie apart) is
    quantized on the way (tensor scale x_scale); W codes [N, K / 2] with tiled scales, tensor scale w_scale.
    residual [M, N] may be out."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.fp4_linear(x, W, w_scales, fmt, x_scale, w_scale, bias, act, out, workspace, residual)
        if got is not None:
            return got
    bf16 = _torch().bfloat16
    f, a = _fp4_format(fmt), _act(act)
    dev = _call_device(x, "x")
    ldx = _row_stride(x, bf16, "x", dev)
    M, K = _tokens(x, a)
    N, Kw, pw, pws = _fp4_operand(W, w_scales, f, "W", dev)
    if Kw != K:
        raise ValueError("x and W must have the same columns")
    pb = None if bias is None else _typed(bias, bf16, "bias", dev, (N,))
    pr = None if residual is None else _typed(residual, bf16, "residual", dev, (M, N))
    y = _out_rows(out, M, N, dev, x.device, stream)
    ws = _given_workspace(workspace, dev) if workspace is not None else fp4_linear_workspace(M, K, fmt, x.device, stream)
    st = lib().ck_fp4_linear(x.data_ptr(), M, K, ldx, a, f, x_scale, pw, pws, w_scale, N, pb, pr, y.data_ptr(),
                             ws.data_ptr(), ws.nbytes, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_fp4_linear")
    return y


def fp4_swiglu_mlp_workspace(M: int, H: int, I: int, fmt: str, device="cuda", stream=None):
    """A workspace for fp4_swiglu_mlp calls of these sizes."""
    n = int(lib().ck_fp4_swiglu_mlp_workspace_bytes(M, H, I, _fp4_format(fmt)))
    return _new_on((max(n, 16),), _torch().uint8, device, stream)


def fp4_swiglu_mlp(x, Wgu, gu_scales, Wd, d_scales, fmt: str, x_scale: float = 1.0, gate_up_scale: float = 1.0,
                   act_scale: float = 1.0, down_scale: float = 1.0, bgu=None, bd=None, residual=None, out=None,
                   workspace=None, stream=None):
    """SwiGLU MLP on 4-bit weights -> bf16 [M, H]: h = linear(x, Wgu [2I, H / 2]), y = linear(silu(gate) * up,
    Wd [H, I / 2]) + residual.  Tensor scales: x_scale of x, act_scale of silu(gate) * up, the others of the
    weights.  residual may be x or out."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.fp4_swiglu_mlp(x, Wgu, gu_scales, Wd, d_scales, fmt, x_scale, gate_up_scale, act_scale, down_scale, bgu,
                                   bd, residual, out, workspace)
        if got is not None:
            return got
    bf16 = _torch().bfloat16
    f = _fp4_format(fmt)
    dev = _call_device(x, "x")
    px = _typed(x, bf16, "x", dev)
    M, H = x.shape
    N, Kw, pgu, pgus = _fp4_operand(Wgu, gu_scales, f, "Wgu", dev)
    Nd, I, pd, pds = _fp4_operand(Wd, d_scales, f, "Wd", dev)
    if Kw != H or Nd != H or N != 2 * I:
        raise ValueError("Wgu must be [2I, H / 2] and Wd [H, I / 2] of x's H columns")
    pbgu, pbd = _typed(bgu, bf16, "bgu", dev, (N,)), _typed(bd, bf16, "bd", dev, (H,))
    pr = _typed(residual, bf16, "residual", dev, (M, H))
    y = _out_rows(out, M, H, dev, x.device, stream)
    ws = (_given_workspace(workspace, dev) if workspace is not None else
          fp4_swiglu_mlp_workspace(M, H, I, fmt, x.device, stream))
    st = lib().ck_fp4_swiglu_mlp(px, M, H, I, f, x_scale, pgu, pgus, gate_up_scale, pbgu, act_scale, pd, pds,
                                 down_scale, pbd, pr, y.data_ptr(), ws.data_ptr(), ws.nbytes, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_fp4_swiglu_mlp")
    return y


def _norm_call(x, branch, post_weight, gate, scale, shift, tokens_per_group, x_factor, branch_factor, norm, weight,
               bias, eps, h_out, stream):
    """What block_norm and block_norm_fp4 share -> (C arguments up to h_out's, h, device)."""
    bf16 = _torch().bfloat16
    dev = _call_device(x, "x")
    ldx = _row_stride(x, bf16, "x", dev)
    shape = x.shape
    T, H = shape
    kind = _NORMS.get(norm)
    if kind is None:
        raise ValueError("norm must be 'rms' or 'layer'")
    pb = pg = psc = psh = pp = pw = pbias = ph = None
    ldb = ldh = 0
    ldm = H
    if branch is not None:
        pb, ldb = branch.data_ptr(), _row_stride(branch, bf16, "branch", dev, shape)
    if gate is not None or scale is not None or shift is not None:
        groups = -(-T // tokens_per_group) if tokens_per_group > 0 else 1
        rows = set()
        for t, what in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
            if t is None:
                continue
            ld = _row_stride(t, bf16, what, dev)
            if t.shape[0] < groups or t.shape[1] != H:
                raise ValueError(f"{what} must have a row of {H} for each of {groups} groups")
            rows.add(ld if groups > 1 else H)
        if len(rows) > 1:
            raise ValueError("gate, scale and shift must have their rows at one stride")
        ldm = rows.pop()
        pg, psc, psh = _ptr(gate), _ptr(scale), _ptr(shift)
    wdt = CK_BF16
    if weight is not None or bias is not None or post_weight is not None:
        dt, wdt = _weight_type(weight, bias, post_weight)
        vector = (H,)
        if weight is not None:
            pw = _typed(weight, dt, "weight", dev, vector)
        if bias is not None:
            pbias = _typed(bias, dt, "bias", dev, vector)
        if post_weight is not None:
            pp = _typed(post_weight, dt, "post_weight", dev, vector)
    if h_out is not None:
        ph, ldh = h_out.data_ptr(), _row_stride(h_out, bf16, "h_out", dev, shape)
    elif branch is not None or x_factor != 1.0:
        h_out, ldh = _new_like(x, stream), H
        ph = h_out.data_ptr()
    else:
        h_out = x  # without a branch and a factor the stream itself is h
    return (x.data_ptr(), ldx, pb, ldb, T, H, pp, pg, psc, psh, ldm, tokens_per_group, x_factor, branch_factor, kind,
            pw, pbias, wdt, eps, ph, ldh), h_out, dev


def block_norm(x, branch=None, post_weight=None, gate=None, x_factor: float = 1.0, branch_factor: float = 1.0,
               norm: str = "rms", weight=None, bias=None, scale=None, shift=None, tokens_per_group: int = 0,
               eps: float = 1e-6, h_out=None, n_out=None, stream=None):
    """The residual sum behind a block and the norm in front of the next, in one pass -> (h, n), bf16 [T, H].

    h = x_factor x + branch_factor gate b, b the branch (RMS-normed times post_weight, where that is given);
    n = norm(h) weight + bias, then n (1 + scale) + shift.  x, branch [T, H] bf16, rows may lie apart; weights
    [H], f32 or bf16 alike; gate, scale, shift bf16 [groups, H], a row for every tokens_per_group tokens (0: one
    row for all).  h_out=x and n_out=branch work in place.  Without a branch and a factor h is x."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.block_norm(x, branch, post_weight, gate, x_factor, branch_factor, norm, weight, bias, scale, shift,
                               tokens_per_group, eps, h_out, n_out)
        if got is not None:
            return got
    args, h, dev = _norm_call(x, branch, post_weight, gate, scale, shift, tokens_per_group, x_factor, branch_factor,
                              norm, weight, bias, eps, h_out, stream)
    if n_out is None:
        n_out, ldn = _new_like(x, stream), args[5]
    else:
        ldn = _row_stride(n_out, x.dtype, "n_out", dev, x.shape)
    st = lib().ck_block_norm(*args, n_out.data_ptr(), ldn, _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_block_norm")
    return h, n_out


def block_norm_fp4(x, branch=None, fmt: str = "nv", n_scale: float = 1.0, post_weight=None, gate=None,
                   x_factor: float = 1.0, branch_factor: float = 1.0, norm: str = "rms", weight=None, bias=None,
                   scale=None, shift=None, tokens_per_group: int = 0, eps: float = 1e-6, h_out=None, codes=None,
                   scales=None, stream=None):
    """block_norm whose n is quantized as by fp4_quantize (tensor scale n_scale) -> (h, codes, tiled scales)."""
    if stream is None and (quick := _quick_module or _quick()) is not None:
        got = quick.block_norm_fp4(x, branch, fmt, n_scale, post_weight, gate, x_factor, branch_factor, norm, weight, bias,
                                   scale, shift, tokens_per_group, eps, h_out, codes, scales)
        if got is not None:
            return got
    u8 = _torch().uint8
    f = _fp4_format(fmt)
    args, h, dev = _norm_call(x, branch, post_weight, gate, scale, shift, tokens_per_group, x_factor, branch_factor,
                              norm, weight, bias, eps, h_out, stream)
    T, H = args[4], args[5]
    if H % 32 != 0:
        raise CkError(CK_ERR_SHAPE, "ck_block_norm_fp4")
    if codes is None:
        codes = _new_on((T, H // 2), u8, x.device, stream)
    scales = _scales_out(scales, _tiled_bytes(f, T, H), dev, x.device, stream)
    st = lib().ck_block_norm_fp4(*args, f, n_scale, _typed(codes, u8, "codes", dev, (T, H // 2)), scales.data_ptr(),
                                 _run_stream(stream, dev))
    if st != CK_OK:
        raise CkError(st, "ck_block_norm_fp4")
    return h, codes, scales


def debug_int8_gemm_s32(xq, Wq, stream=None):
    """Raw int32 accumulators of the GEMM engine (test hook)."""
    torch = _torch()
    _require_cuda(xq, Wq)
    M, K = xq.shape
    N = Wq.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    ws = _workspace(workspace_bytes(CK_OP_DEBUG_GEMM_S32, M, K, N), xq.device)
    _check(lib().ck_debug_int8_gemm_s32(xq.data_ptr(), Wq.data_ptr(), M, N, K, acc.data_ptr(),
                                        ws.data_ptr(), ws.numel(), _stream(stream)),
           "ck_debug_int8_gemm_s32")
    return acc


def debug_gemv_s32(xq, Wpacked, wlayout: int, N: int, stream=None):
    """Exact int32 sums of the small-M GEMV engines on INT8 codes xq [M, K] and a
    GEMV-resident weight (test hook): the weight codes as the engines see them
    on the INT8 grid (6- / 4-bit codes times 4 / 16)."""
    torch = _torch()
    _require_cuda(xq, Wpacked)
    M, K = xq.shape
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    _check(lib().ck_debug_gemv_s32(xq.data_ptr(), M, K, Wpacked.data_ptr(), wlayout, N,
                                   acc.data_ptr(), _stream(stream)), "ck_debug_gemv_s32")
    return acc


def poll_device_status(stream=None) -> int:
    """Synchronize the stream; CK_OK, CK_ERR_TIMEOUT or CK_ERR_INDEX from the device status word."""
    return int(lib().ck_poll_device_status(_stream(stream)))


def set_wait_timeout_ns(ns: int) -> None:
    lib().ck_set_wait_timeout_ns(int(ns))


def set_launch_overlap(on: bool) -> None:
    """Overlapped launches across calls (ck_set_launch_overlap): the GEMM / GEMV
    may read the weight operands before the work ahead of it on the stream has
    finished, so those weights must be settled (prepared, then synchronized)."""
    lib().ck_set_launch_overlap(1 if on else 0)


def debug_gemm_tile_choice(M: int, N: int, K: int, sms: int) -> int:
    """The GEMM tile code the engine picks for M x K -> N on a GPU of sms SMs (host only)."""
    return int(lib().ck_debug_gemm_tile_choice(int(M), int(N), int(K), int(sms)))


def debug_force_gemm_tile(bn: int) -> None:
    """Force the GEMM tile width (64/128/256); 0 restores the automatic choice."""
    lib().ck_debug_force_gemm_tile(int(bn))


def debug_force_gemv_quantizer(mode: int) -> None:
    """1: quantizer kernel + GEMV, 2: quantize inside the GEMV's CTAs where the
    shape allows; 0 restores the automatic choice."""
    lib().ck_debug_force_gemv_quantizer(int(mode))


def debug_stalled_wait(stream=None) -> int:
    return int(lib().ck_debug_stalled_wait(_stream(stream)))

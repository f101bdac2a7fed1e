"""The 4-bit operators and the block norm without a GPU: sizes, and refusals
before anything touches the device (the fake pointers are never followed)."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck

P = 0x10000
BIG = 1 << 40
MX, NV = ck.CK_FP4_MX, ck.CK_FP4_NV
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    ck.build()
    return ck.lib()


def test_scale_bytes(L):
    assert L.ck_fp4_scale_bytes(NV, 1, 32) == 512
    assert L.ck_fp4_scale_bytes(NV, 128, 64) == 512
    assert L.ck_fp4_scale_bytes(NV, 129, 96) == 2 * 2 * 512
    assert L.ck_fp4_scale_bytes(MX, 129, 96) == 2 * 512
    assert L.ck_fp4_scale_bytes(MX, 300, 160) == 3 * 2 * 512
    for bad in ((2, 1, 32), (NV, 0, 32), (NV, 1, 0), (NV, 1, 48), (MX, 1, 32768 + 32), (MX, 1 << 31, 32)):
        assert L.ck_fp4_scale_bytes(*bad) == 0


def test_workspace_bytes(L):
    n = L.ck_fp4_linear_workspace_bytes(100, 96, NV)
    assert n >= 100 * 48 + L.ck_fp4_scale_bytes(NV, 100, 96)
    assert L.ck_fp4_linear_workspace_bytes(100, 97, NV) == 0
    assert L.ck_fp4_linear_workspace_bytes(0, 96, NV) == 0
    assert L.ck_fp4_linear_workspace_bytes(100, 96, 3) == 0
    m = L.ck_fp4_swiglu_mlp_workspace_bytes(100, 96, 64, MX)
    assert m >= 100 * 48 + 100 * 2 * 64 * 2 + 100 * 32
    assert L.ck_fp4_swiglu_mlp_workspace_bytes(100, 96, 60, MX) == 0


def test_reference_tiles_by_hand():
    """Row 70, block 9 of 12 (NV, K = 192: three words): tile 0, word 2, byte 1 of the row's word."""
    s = np.zeros((130, 12), np.uint8)
    s[70, 9] = 1
    s[129, 0] = 2
    t = ref.tile(s, "nv")
    assert t.size == 2 * 3 * 512
    assert t[2 * 512 + 16 * (70 % 32) + 4 * (70 // 32) + 1] == 1
    assert t[3 * 512 + 16 * 1] == 2
    assert np.count_nonzero(t) == 2
    assert np.array_equal(ref.untile(t, 130, 192, "nv"), s)


def test_reference_codes_by_hand():
    q = np.array([0.0, 0.25, 0.2500001, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 9.0, -0.75, -5.0])
    assert ref.e2m1(q).tolist() == [0, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 10, 14]
    assert ref.e4m3(np.array([448.0, 500.0, 1.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 1.5 * 2 ** -9, 2.0 ** -6])).tolist() == \
        [0x7e, 0x7e, 0x38, 0x38, 0x3a, 1, 0, 2, 8]
    every = np.arange(127, dtype=np.uint8)
    assert np.array_equal(ref.e4m3(ref.e4m3_value(every)), every)
    assert torch.equal(torch.from_numpy(ref.e4m3_value(every)).float(), torch.from_numpy(every).view(torch.float8_e4m3fn).float())
    codes, scales = ref.quantize(np.array([[6.0] + [0.75] * 31]), "mx")
    assert scales.tolist() == [[127]] and codes[0, :2].tolist() == [7, 2]


def quantize(L, **kw):
    a = dict(x=P, xdt=ck.CK_BF16, M=4, K=64, ldx=64, act=0, fmt=NV, t=0.5, codes=P, scales=P, s=None)
    a.update(kw)
    return L.ck_fp4_quantize(*a.values())


def test_quantize_refusals(L):
    for p in ("x", "codes", "scales"):
        assert quantize(L, **{p: None}) == ck.CK_ERR_NULL
        assert quantize(L, **{p: P + 8}) == ck.CK_ERR_ALIGN
    for kw in (dict(fmt=2), dict(fmt=-1), dict(act=2), dict(t=0.0), dict(t=-1.0), dict(t=INF), dict(t=NAN), dict(t=2.0 ** 61),
               dict(t=2.0 ** -61), dict(fmt=MX, t=0.5)):
        assert quantize(L, **kw) == ck.CK_ERR_INVALID, kw
    assert quantize(L, xdt=2) == ck.CK_ERR_DTYPE
    assert quantize(L, xdt=ck.CK_F32, act=1, ldx=128) == ck.CK_ERR_DTYPE
    for kw in (dict(M=0), dict(M=1 << 31), dict(K=0), dict(K=48), dict(K=32800, ldx=32800), dict(ldx=56), dict(ldx=68),
               dict(act=1, ldx=120), dict(xdt=ck.CK_F32, ldx=66)):
        assert quantize(L, **kw) == ck.CK_ERR_SHAPE, kw


def test_tile_scales_refusals(L):
    assert L.ck_fp4_tile_scales(None, 4, 64, NV, P, None) == ck.CK_ERR_NULL
    assert L.ck_fp4_tile_scales(P, 4, 64, NV, None, None) == ck.CK_ERR_NULL
    assert L.ck_fp4_tile_scales(P, 4, 64, 5, P, None) == ck.CK_ERR_INVALID
    assert L.ck_fp4_tile_scales(P, 4, 40, NV, P, None) == ck.CK_ERR_SHAPE
    assert L.ck_fp4_tile_scales(P, 4, 64, NV, P + 4, None) == ck.CK_ERR_ALIGN


def gemm(L, **kw):
    a = dict(codes=P, scales=P, M=4, K=64, fmt=NV, W=P, ws=P, N=16, alpha=1.0, bias=None, residual=None, y=P, s=None)
    a.update(kw)
    return L.ck_fp4_gemm(*a.values())


def test_gemm_refusals(L):
    for p in ("codes", "scales", "W", "ws", "y"):
        assert gemm(L, **{p: None}) == ck.CK_ERR_NULL
    for p in ("codes", "scales", "W", "ws", "y", "bias", "residual"):
        assert gemm(L, **{p: P + 2}) == ck.CK_ERR_ALIGN
    for kw in (dict(fmt=9), dict(alpha=INF), dict(alpha=NAN)):
        assert gemm(L, **kw) == ck.CK_ERR_INVALID
    for kw in (dict(M=0), dict(K=16), dict(K=72), dict(N=0), dict(N=12), dict(N=1 << 31)):
        assert gemm(L, **kw) == ck.CK_ERR_SHAPE


def linear(L, **kw):
    a = dict(x=P, M=4, K=64, ldx=64, act=0, fmt=NV, xt=0.5, W=P, ws=P, wt=0.5, N=16, bias=None, residual=None, y=P, work=P,
             bytes=BIG, s=None)
    a.update(kw)
    return L.ck_fp4_linear(*a.values())


def test_linear_refusals(L):
    for p in ("x", "W", "ws", "y"):
        assert linear(L, **{p: None}) == ck.CK_ERR_NULL
    for p in ("x", "W", "ws", "y", "bias", "residual", "work"):
        assert linear(L, **{p: P + 4}) == ck.CK_ERR_ALIGN
    for kw in (dict(fmt=9), dict(act=3), dict(xt=0.0), dict(wt=NAN), dict(fmt=MX, xt=1.0, wt=0.5)):
        assert linear(L, **kw) == ck.CK_ERR_INVALID
    for kw in (dict(M=0), dict(K=80, ldx=80), dict(ldx=60), dict(act=1), dict(N=4)):
        assert linear(L, **kw) == ck.CK_ERR_SHAPE
    assert linear(L, work=None) == ck.CK_ERR_WORKSPACE
    assert linear(L, bytes=L.ck_fp4_linear_workspace_bytes(4, 64, NV) - 1) == ck.CK_ERR_WORKSPACE


def mlp(L, **kw):
    a = dict(x=P, M=4, H=64, I=96, fmt=NV, xt=0.5, gu=P, gus=P, gut=0.5, bgu=None, at=0.5, d=P, ds=P, dt=0.5, bd=None,
             residual=None, y=P, work=P, bytes=BIG, s=None)
    a.update(kw)
    return L.ck_fp4_swiglu_mlp(*a.values())


def test_mlp_refusals(L):
    for p in ("x", "gu", "gus", "d", "ds", "y"):
        assert mlp(L, **{p: None}) == ck.CK_ERR_NULL
    for p in ("x", "gu", "gus", "d", "ds", "y", "bgu", "bd", "residual", "work"):
        assert mlp(L, **{p: P + 4}) == ck.CK_ERR_ALIGN
    for kw in (dict(fmt=9), dict(xt=0.0), dict(gut=INF), dict(at=-1.0), dict(dt=NAN), dict(fmt=MX)):
        assert mlp(L, **kw) == ck.CK_ERR_INVALID
    for kw in (dict(M=0), dict(H=72), dict(I=40), dict(I=0)):
        assert mlp(L, **kw) == ck.CK_ERR_SHAPE
    assert mlp(L, work=None) == ck.CK_ERR_WORKSPACE
    assert mlp(L, bytes=L.ck_fp4_swiglu_mlp_workspace_bytes(4, 64, 96, NV) - 1) == ck.CK_ERR_WORKSPACE


NORM = dict(x=P, ldx=64, branch=P, ldb=64, T=4, H=64, post=None, gate=None, scale=None, shift=None, ldm=64, per=0, xf=1.0,
            bf=1.0, norm=0, weight=None, bias=None, wdt=ck.CK_BF16, eps=1e-6, h=P, ldh=64)


def norm(L, n=P, ldn=64, **kw):
    return L.ck_block_norm(*{**NORM, **kw}.values(), n, ldn, None)


def norm_fp4(L, fmt=NV, t=0.5, codes=P, scales=P, **kw):
    return L.ck_block_norm_fp4(*{**NORM, **kw}.values(), fmt, t, codes, scales, None)


def test_block_norm_refusals(L):
    for call in (norm, norm_fp4):
        assert call(L, x=None) == ck.CK_ERR_NULL
        assert call(L, branch=None, gate=P) == ck.CK_ERR_NULL
        assert call(L, branch=None, post=P) == ck.CK_ERR_NULL
        for p in ("x", "branch", "post", "gate", "scale", "shift", "weight", "bias", "h"):
            assert call(L, **{p: P + 8}) == ck.CK_ERR_ALIGN
        for kw in (dict(norm=2), dict(xf=INF), dict(bf=NAN), dict(eps=-1.0), dict(eps=NAN)):
            assert call(L, **kw) == ck.CK_ERR_INVALID, kw
        assert call(L, wdt=3) == ck.CK_ERR_DTYPE
        for kw in (dict(T=0), dict(T=1 << 31), dict(H=0), dict(H=20), dict(H=16384 + 8, ldx=20000, ldb=20000, ldh=20000),
                   dict(ldx=56), dict(ldx=68), dict(ldb=0), dict(ldh=8), dict(per=-1), dict(per=2, gate=P, ldm=32)):
            assert call(L, **kw) == ck.CK_ERR_SHAPE, kw
    assert norm(L, n=None) == ck.CK_ERR_NULL
    assert norm(L, n=P + 4) == ck.CK_ERR_ALIGN
    assert norm(L, ldn=60) == ck.CK_ERR_SHAPE
    assert norm_fp4(L, codes=None) == ck.CK_ERR_NULL
    assert norm_fp4(L, scales=None) == ck.CK_ERR_NULL
    assert norm_fp4(L, codes=P + 4) == ck.CK_ERR_ALIGN
    assert norm_fp4(L, fmt=2) == ck.CK_ERR_INVALID
    assert norm_fp4(L, t=0.0) == ck.CK_ERR_INVALID
    assert norm_fp4(L, H=40) == ck.CK_ERR_SHAPE

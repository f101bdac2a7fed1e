"""Sizes at which a product of 4-bit floats is refused, without a GPU (the fake pointers are never followed)."""
import pytest

import swiglu_mlp_group_gb300 as ck
from test_fp4_devices import calls  # noqa: F401 (a fixture)

P, BIG = 0x10000, 1 << 60
NV = ck.CK_FP4_NV


@pytest.fixture(scope="module")
def L():
    ck.build()
    return ck.lib()


@pytest.mark.parametrize("M", [33, 1000])
@pytest.mark.parametrize("N", [(1 << 31) - 376, (1 << 31) - 8])
def test_columns_that_a_tile_cannot_count(M, N, L):
    """Products of many tokens work on tiles of up to 384 columns and count those past N in 32 bits, too."""
    assert L.ck_fp4_gemm(P, P, M, 32, NV, P, P, N, 1.0, P, P, P, None) == ck.CK_ERR_SHAPE
    assert L.ck_fp4_linear(P, M, 32, 32, 0, NV, 1.0, P, P, 1.0, N, P, P, P, P, BIG, None) == ck.CK_ERR_SHAPE


def test_odd_columns_are_not_halved(calls):
    """[gate | up] has an even number of columns; of 2K + 1 the last would be left out without a word."""
    from test_attention_devices import Stub
    U8 = ck._torch().uint8
    M, K, N = 5, 64, 24

    def x(cols):
        s = Stub((M, cols))
        s.stride = lambda: (4 * K, 1)
        return s
    scales = Stub((512,), U8)
    for cols, ok in ((2 * K, True), (2 * K + 1, False)):
        for call in (lambda: ck.fp4_quantize(x(cols), "nv", act="swiglu", codes=Stub((M, K // 2), U8), scales=scales),
                     lambda: ck.fp4_linear(x(cols), Stub((N, K // 2), U8), scales, "nv", act="swiglu", out=Stub((M, N)),
                                           workspace=Stub((1 << 20,), U8))):
            calls.clear()
            if ok:
                call()
                assert len(calls) == 1
            else:
                with pytest.raises(ValueError):
                    call()
                assert not calls

"""Sizes at which a product of 4-bit floats is refused, without a GPU (the fake pointers are never followed)."""
import pytest

import swiglu_mlp_group_gb300 as ck

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

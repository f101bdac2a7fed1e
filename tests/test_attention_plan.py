"""The division of attention's work as its workspace sizes show it, without a GPU."""
import time

import pytest

import swiglu_mlp_group_gb300 as ck


@pytest.fixture(scope="module")
def L():
    ck.build()
    return ck.lib()


# key heads x row tiles near the number of SMs: the smallest chunk of key tiles for which every item has an SM of its own
# is then as long as the prefix
@pytest.mark.parametrize("B,Hq,H", [(18, 8, 8), (143, 1, 1)])
def test_long_prefixes_are_planned_at_once(L, B, Hq, H):
    best = 1e9
    for _ in range(5):
        t = time.perf_counter()
        assert L.ck_prefix_attention_workspace_bytes(B, 1, Hq, H, 128, 1 << 30, 4096) > 0
        best = min(best, time.perf_counter() - t)
    assert best < 1e-3, f"{best * 1e6:.0f} us"  # some 2 us of arithmetic; tile by tile it is 5 to 50 ms


# what the binding allocates and what the call asks for are one
@pytest.mark.parametrize("sizes", [(64, 1, 32, 8, 128, 8192, 1024), (4, 1, 32, 8, 128, 1000, 130),
                                   (128, 1, 64, 8, 128, 32768, 4096), (1, 2048, 8, 2, 128, 0, 2048)])
def test_a_workspace_short_of_a_byte_is_refused(L, sizes):
    P = 0x10000
    B, Lq, Hq, H, D, plen, mlen = sizes
    need = L.ck_prefix_attention_workspace_bytes(*sizes)
    assert need > 0

    def call(ws, n):
        return L.ck_prefix_attention(P, Hq * D, B, Lq, Hq, H, D, P, P, 4096, 16, P, plen, P, 2048, P, mlen, 0.1, P, Hq * D,
                                     ws, n, None)

    assert call(P, need - 1) == ck.CK_ERR_WORKSPACE
    assert call(None, need) == ck.CK_ERR_WORKSPACE
    assert call(P + 8, need) == ck.CK_ERR_ALIGN


def test_a_cross_workspace_short_of_a_byte_is_refused(L):
    P = 0x10000
    for B, Lq, Lk, Hq, H in ((1, 1, 8192, 8, 8), (1, 300, 9000, 4, 4)):
        need = L.ck_cross_attention_workspace_bytes(B, Lq, Lk, Hq, H, 128)
        assert need > 0
        for ws, n in ((P, need - 1), (None, need)):
            assert L.ck_cross_attention(P, Hq * 128, P, H * 128, P, H * 128, B, Lq, Lk, Hq, H, 128, P, 0.1, P, Hq * 128, ws,
                                        n, None) == ck.CK_ERR_WORKSPACE


# a call without lengths may be cut another way; it asks for no more than the size function says
@pytest.mark.parametrize("B,Lq,Lk,Hq,H", [(21, 1, 2300, 8, 8), (23, 20, 2100, 8, 8), (2, 1300, 4300, 14, 14),
                                          (40, 1, 5000, 4, 4), (1, 1, 8192, 8, 8)])
def test_even_calls_need_no_more(L, B, Lq, Lk, Hq, H):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake pointers must not reach a GPU")
    P = 0x10000
    need = L.ck_cross_attention_workspace_bytes(B, Lq, Lk, Hq, H, 128)
    for lens in (None, P):
        assert L.ck_cross_attention(P, Hq * 128, P, H * 128, P, H * 128, B, Lq, Lk, Hq, H, 128, lens, 0.1, P, Hq * 128, P,
                                    need, None) == ck.CK_ERR_UNSUPPORTED_DEVICE

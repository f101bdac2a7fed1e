"""The attention entry points without a GPU: every refusal, checked before any
pointer is used, and the binding's own checks of tensors."""
import pytest
import torch

import swiglu_mlp_group_gb300 as ck

P = 0x10000  # a fake, 16-byte aligned device address


@pytest.fixture(scope="module")
def L():
    ck.build()
    return ck.lib()


def norm_rope(L, **kw):
    a = dict(q=P, ldq=512, Hq=4, wq=P, k=P, ldk=512, Hk=2, wk=P, wdt=ck.CK_BF16, T=3, D=128, eps=1e-6, cs=P,
             max_pos=100, rot=128, mode=0, pos=P, qo=P, ldqo=512, ko=P, ldko=256, s=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ck_qk_norm_rope(*a.values())


def append(L, **kw):
    a = dict(k=P, ldk=256, v=P, ldv=256, T=3, H=2, D=128, wk=P, wdt=ck.CK_BF16, eps=1e-6, cs=P, max_pos=100, rot=128,
             mode=0, pos=P, slots=P, kc=P, vc=P, pages=10, page=16, s=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ck_kv_append(*a.values())


def prefix(L, **kw):
    a = dict(q=P, ldq=1024, B=2, Lq=1, Hq=8, H=2, D=128, kc=P, vc=P, pages=100, page=16, pp=P, plen=50, bt=P,
             stride=4, lens=P, mlen=64, scale=0.1, out=P, ldo=1024, ws=P, wsb=1 << 40, s=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ck_prefix_attention(*a.values())


def cross(L, **kw):
    a = dict(q=P, ldq=1024, k=P, ldk=256, v=P, ldv=256, B=2, Lq=5, Lk=70, Hq=8, H=2, D=128, lens=P, scale=0.1, out=P,
             ldo=1024, ws=P, wsb=1 << 40, s=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ck_cross_attention(*a.values())


NULLS = [(norm_rope, ["q", "k", "qo", "ko", "cs", "pos"]), (append, ["k", "v", "slots", "kc", "vc", "cs", "pos"]),
         (prefix, ["q", "kc", "vc", "pp", "bt", "lens", "out"]), (cross, ["q", "k", "v", "out"])]


@pytest.mark.parametrize("call,name", [(c, n) for c, ns in NULLS for n in ns])
def test_null_pointers(L, call, name):
    assert call(L, **{name: None}) == ck.CK_ERR_NULL


ALIGNED = [(norm_rope, ["q", "k", "qo", "ko", "wq", "wk", "cs"]), (append, ["k", "v", "wk", "cs", "kc", "vc"]),
           (prefix, ["q", "kc", "vc", "out"]), (cross, ["q", "k", "v", "out"])]


@pytest.mark.parametrize("call,name", [(c, n) for c, ns in ALIGNED for n in ns])
def test_alignment(L, call, name):
    assert call(L, **{name: P + 8}) == ck.CK_ERR_ALIGN


SHAPES = [
    (norm_rope, [dict(T=0), dict(T=-1), dict(D=120), dict(D=8), dict(D=272), dict(rot=8), dict(rot=144), dict(rot=-16),
                 dict(max_pos=0), dict(Hq=0), dict(ldq=504), dict(ldq=516), dict(ldk=248), dict(ldqo=256),
                 dict(ldko=128), dict(T=1 << 40), dict(T=1 << 30), dict(Hk=-1)]),
    (append, [dict(T=0), dict(D=100), dict(rot=160), dict(H=0), dict(pages=0), dict(page=0), dict(page=65537),
              dict(ldk=128), dict(ldv=260), dict(max_pos=1 << 40)]),
    (prefix, [dict(B=0), dict(Lq=0), dict(Hq=0), dict(H=0), dict(Hq=9), dict(D=96), dict(D=256), dict(page=8),
              dict(page=48), dict(page=256), dict(pages=0), dict(pages=1 << 31), dict(pages=1 << 27), dict(plen=-1),
              dict(mlen=-1), dict(mlen=65), dict(stride=0), dict(ldq=1016), dict(ldq=1028), dict(ldo=512),
              dict(B=1 << 40), dict(B=1 << 30, Lq=4), dict(Hq=258, H=2, ldq=1 << 16, ldo=1 << 16)]),
    (cross, [dict(B=0), dict(Lq=0), dict(Lk=-1), dict(Hq=0), dict(Hq=7), dict(D=32), dict(ldq=8), dict(ldk=128),
             dict(ldv=257), dict(ldo=1000), dict(Lk=1 << 31), dict(B=4, Lk=1 << 30)]),
]


@pytest.mark.parametrize("call,kw", [(c, kw) for c, ks in SHAPES for kw in ks])
def test_sizes(L, call, kw):
    assert call(L, **kw) == ck.CK_ERR_SHAPE


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
def test_scale(L, bad):
    assert prefix(L, scale=bad) == ck.CK_ERR_INVALID
    assert cross(L, scale=bad) == ck.CK_ERR_INVALID


def test_other_arguments(L):
    for call in (norm_rope, append):
        assert call(L, mode=2) == ck.CK_ERR_INVALID
        assert call(L, eps=-1e-6) == ck.CK_ERR_INVALID
        assert call(L, eps=float("nan")) == ck.CK_ERR_INVALID
        assert call(L, wdt=7) == ck.CK_ERR_DTYPE


def test_good_arguments_reach_the_device_check(L):
    if torch.cuda.is_available():
        pytest.skip("the fake pointers must not reach a GPU")
    for call in (norm_rope, append, prefix, cross):
        assert call(L) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert norm_rope(L, k=None, Hk=0, ko=None) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert norm_rope(L, cs=None, rot=0, pos=None, wq=None, wk=None) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert prefix(L, plen=0, pp=None) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert prefix(L, mlen=0, bt=None, lens=None, stride=0) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert cross(L, Lk=0, k=None, v=None, ldk=0, ldv=0) == ck.CK_ERR_UNSUPPORTED_DEVICE
    assert cross(L, lens=None) == ck.CK_ERR_UNSUPPORTED_DEVICE


def test_workspace(L):
    """A workspace that is too small is refused; sizes that the calls refuse have none."""
    need = L.ck_prefix_attention_workspace_bytes(64, 1, 32, 8, 128, 8192, 1024)
    if need > 0:
        assert prefix(L, B=64, Hq=32, H=8, ldq=4096, ldo=4096, plen=8192, mlen=1024, stride=64,
                      wsb=need - 1) == ck.CK_ERR_WORKSPACE
        assert prefix(L, B=64, Hq=32, H=8, ldq=4096, ldo=4096, plen=8192, mlen=1024, stride=64,
                      ws=None) == ck.CK_ERR_WORKSPACE
    need = L.ck_cross_attention_workspace_bytes(1, 1, 8192, 8, 8, 128)
    if need > 0:
        assert cross(L, B=1, Lq=1, Lk=8192, H=8, ldk=1024, ldv=1024, wsb=need - 1) == ck.CK_ERR_WORKSPACE
    assert L.ck_prefix_attention_workspace_bytes(0, 1, 32, 8, 128, 10, 10) == 0
    assert L.ck_prefix_attention_workspace_bytes(1, 1, 30, 8, 128, 10, 10) == 0
    assert L.ck_cross_attention_workspace_bytes(1, 1, -1, 8, 8, 128) == 0


def test_status_name():
    assert ck.status_string(ck.CK_ERR_INDEX).startswith("CK_ERR_INDEX")


def test_binding_refuses_other_tensors():
    """Host tensors, other types and layouts never reach the library."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ck.qk_norm_rope(x, x)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ck.kv_append(x, x, cache, cache, torch.arange(4))
    with pytest.raises(ValueError):
        ck.prefix_attention(x[None], cache, cache, None, 0, None, None, 0)
    with pytest.raises(ValueError):
        ck.cross_attention(x[None], x[None], x[None, :2])

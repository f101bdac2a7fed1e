"""Head norms with the position rotation, and the append to a paged cache,
against their definitions in 64 bits."""
import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

EPS = 1e-5


def case(seed, T, Hq, Hk, D, rot, wdtype=torch.bfloat16, max_pos=500):
    dev = device()
    g = ref.gen(seed)
    packed = ref.randn(g, T, (Hq + 2 * Hk) * D, std=3.0).to(dev)
    q = packed[:, :Hq * D].view(T, Hq, D)
    k = packed[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    wq, wk = (ref.randn(g, D, dtype=wdtype).to(dev) for _ in range(2))
    table = ref.rope_table(max_pos, rot).to(dev) if rot else None
    pos = torch.randint(0, max_pos, (T,), generator=g).to(torch.int32).to(dev)
    return packed, q, k, wq, wk, table, pos


def reference(x, w, table, pos, mode):
    return ref.norm_rope(x.cpu(), None if w is None else w.cpu(), EPS, None if table is None else table.cpu(),
                         pos.cpu(), mode)


@pytest.mark.parametrize("mode", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(16, 16), (48, 32), (64, 64), (64, 16), (80, 80), (96, 48), (128, 128), (128, 64),
                                   (176, 160), (256, 256), (256, 128), (128, 0)])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (37, 5, 2)])
def test_norm_rope(T, Hq, Hk, D, rot, mode):
    _, q, k, wq, wk, table, pos = case(D + rot, T, Hq, Hk, D, rot)
    qo, ko = ck.qk_norm_rope(q, k, table, pos if rot else None, wq=wq, wk=wk, eps=EPS, mode=mode)
    poll_ok()
    ref.assert_norm_rope(qo, reference(q, wq, table, pos, mode), "q")
    ref.assert_norm_rope(ko, reference(k, wk, table, pos, mode), "k")


@pytest.mark.parametrize("mode", ["half", "interleaved"])
def test_parts_left_out(mode):
    """f32 weights; the norm of one side only; rotation alone; queries alone."""
    _, q, k, wq, wk, table, pos = case(3, 50, 4, 2, 128, 128, wdtype=torch.float32)
    qo, ko = ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=None, eps=EPS, mode=mode)
    ref.assert_norm_rope(qo, reference(q, wq, table, pos, mode))
    ref.assert_norm_rope(ko, reference(k, None, table, pos, mode))
    alone, none = ck.qk_norm_rope(q, None, table, pos, wq=wq, eps=EPS, mode=mode)
    assert none is None and torch.equal(alone, qo)
    qr, kr = ck.qk_norm_rope(q, k, table, pos, mode=mode)
    ref.assert_norm_rope(qr, reference(q, None, table, pos, mode))
    assert torch.equal(kr, ko)
    same, _ = ck.qk_norm_rope(q, k)  # neither: a copy
    assert torch.equal(same, q)
    poll_ok()


def test_in_place_and_strided_outputs():
    packed, q, k, wq, wk, table, pos = case(4, 33, 6, 2, 64, 32)
    want_q, want_k = ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk, eps=EPS)
    wide = torch.full((33, 8 * 64 + 8), 5.0, dtype=torch.bfloat16, device=q.device)
    qo, ko = wide[:, :6 * 64].view(33, 6, 64), wide[:, 6 * 64:8 * 64].view(33, 2, 64)
    ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk, eps=EPS, q_out=qo, k_out=ko)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k) and (wide[:, 512:] == 5).all()
    v = packed[:, 8 * 64:].clone()
    ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk, eps=EPS, q_out=q, k_out=k)
    poll_ok()
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(packed[:, 8 * 64:], v)


def test_extreme_rows():
    """Rows of zeros (eps alone under the root), of tiny and of huge values."""
    _, q, k, wq, wk, table, pos = case(5, 4, 2, 1, 128, 128)
    q, k = q.contiguous(), k.contiguous()
    q[0], q[1], q[2] = 0, q[1] * 2.0 ** -60, q[2] * 2.0 ** 40
    qo, _ = ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk, eps=EPS)
    poll_ok()
    assert (qo[0] == 0).all()
    ref.assert_norm_rope(qo, reference(q, wq, table, pos, "half"))


def test_positions_out_of_range():
    _, q, k, wq, wk, table, pos = case(6, 9, 3, 2, 64, 64)
    want_q, want_k = ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk)
    poll_ok()
    bad = pos.clone()
    bad[2], bad[5] = 500, -1
    qo, ko = torch.full_like(want_q, 9.0), torch.full_like(want_k, 9.0)
    ck.qk_norm_rope(q, k, table, bad, wq=wq, wk=wk, q_out=qo, k_out=ko)
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    keep = torch.tensor([t for t in range(9) if t not in (2, 5)], device=q.device)
    assert torch.equal(qo[keep], want_q[keep]) and torch.equal(ko[keep], want_k[keep])
    assert (qo[[2, 5]] == 9).all() and (ko[[2, 5]] == 9).all()  # not written


@pytest.mark.parametrize("T,H,D,rot,page,mode", [
    (1, 1, 64, 64, 16, "half"), (50, 3, 128, 128, 16, "half"), (333, 8, 128, 64, 64, "interleaved"),
    (77, 2, 96, 96, 1, "interleaved"), (200, 5, 80, 0, 7, "half"), (40, 2, 256, 256, 100, "half"),
    (5, 4, 16, 16, 65536, "half")])
def test_append(T, H, D, rot, page, mode):
    dev = device()
    _, q, k, _, wk, table, pos = case(T, T, H, H, D, rot)
    v = q  # strided values of another place
    pages = -(-T // page) + 2
    kc = torch.full((pages, H, page, D), 3.0, dtype=torch.bfloat16, device=dev)
    vc = torch.full_like(kc, 4.0)
    slots = torch.randperm(pages * page, generator=ref.gen(T))[:T].to(dev)
    slots[T // 2] = -1 if T > 1 else slots[0]
    ck.kv_append(k, v, kc, vc, slots, table, pos if rot else None, wk=wk, eps=EPS, mode=mode)
    poll_ok()
    want_k = reference(k, wk, table, pos, mode)
    keep = (slots >= 0).cpu()
    at = slots.cpu()[keep]
    got_k = kc.transpose(1, 2).reshape(pages * page, H, D).cpu()
    got_v = vc.transpose(1, 2).reshape(pages * page, H, D).cpu()
    ref.assert_norm_rope(got_k[at], want_k[keep])
    assert torch.equal(got_v[at], v.cpu()[keep])
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at] = False
    assert (got_k[rest] == 3).all() and (got_v[rest] == 4).all()  # nothing else is touched


def test_append_is_norm_rope():
    """The append's keys are the same bits as the standalone pass's."""
    dev = device()
    _, q, k, wq, wk, table, pos = case(8, 60, 4, 4, 128, 128)
    _, want = ck.qk_norm_rope(q, k, table, pos, wq=wq, wk=wk, eps=EPS)
    kc, vc = (torch.zeros(4, 4, 16, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ck.kv_append(k, q, kc, vc, torch.arange(60, device=dev), table, pos, wk=wk, eps=EPS)
    poll_ok()
    assert torch.equal(kc.transpose(1, 2).reshape(64, 4, 128)[:60], want)


def test_append_indexes_out_of_range():
    dev = device()
    _, q, k, _, wk, table, pos = case(9, 6, 2, 2, 64, 64)
    kc, vc = (torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    slots = torch.tensor([0, 32, 1 << 40, 3, -(1 << 40), 5], device=dev)
    pos[3] = 500
    ck.kv_append(k, q, kc, vc, slots, table, pos, wk=wk)
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    used = (vc.transpose(1, 2).reshape(32, -1) != 0).any(1).nonzero()[:, 0].tolist()
    assert used == [0, 5]

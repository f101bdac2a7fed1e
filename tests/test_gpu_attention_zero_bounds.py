"""Bounds of zero: no states with pointers all the same, lengths given where none is allowed."""
import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ld", [0, 256])
@pytest.mark.parametrize("Lq", [1, 300])
def test_no_states_behind_real_pointers(Lq, ld):
    """k and v may point somewhere when Lk is 0; nothing of them is read."""
    dev = device()
    q = ref.randn(ref.gen(1), 2, Lq, 4, 64).to(dev)
    kv = torch.full((8, 256), float("nan"), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 7.0)
    st = ck.lib().ck_cross_attention(q.data_ptr(), 256, kv.data_ptr(), ld, kv.data_ptr(), ld, 2, Lq, 0, 4, 4, 64, None,
                                     0.125, out.data_ptr(), 256, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == ck.CK_OK
    poll_ok()
    assert (out == 0).all()


@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("Lq", [1, 3, 300])
def test_lengths_above_a_bound_of_zero(Lq, prefix):
    """As above any other bound: taken as the bound, and reported."""
    dev = device()
    c = ref.Paged(2, 2, 2, 64, 16, prefix, [0, 0]).to(dev)
    q = ref.randn(ref.gen(3), 2, Lq, 4, 64).to(dev)

    def run(seq_lens):
        return ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, prefix, c.block_table, seq_lens, 0)

    good = run(torch.zeros(2, dtype=torch.int32, device=dev))
    poll_ok()
    out = run(torch.tensor([0, 1], dtype=torch.int32, device=dev))
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    assert torch.equal(out, good) and torch.equal(run(None), good)
    poll_ok()
    none = torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device=dev)
    assert (ck.cross_attention(q, none, none, kv_lens=torch.tensor([0, 5], dtype=torch.int32, device=dev)) == 0).all()
    assert ck.poll_device_status() == ck.CK_ERR_INDEX

"""A wait that runs out inside the attention kernel: the call gives up, the status
word says so, and the device is as usable as before.  The wait is made to run out
by a short limit and much to read before the first item is known."""
import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

D, PAGE, TOP, SOME = 64, 128, 2200, 60


def many_empty(B):
    """B sequences behind no prefix, all but the first SOME without tokens: arguments of a call, and its sequences."""
    dev = device()
    lens = [(97 * b) % TOP + 1 for b in range(SOME)]
    c = ref.Paged(50, SOME, 1, D, PAGE, 0, lens, max_len=TOP).to(dev)
    table = torch.zeros(B, c.block_table.shape[1], dtype=torch.int32, device=dev)
    table[:SOME] = c.block_table
    seq_lens = torch.zeros(B, dtype=torch.int32, device=dev)
    seq_lens[:SOME] = c.seq_lens
    q = torch.zeros(B, 1, 2, D, dtype=torch.bfloat16, device=dev)
    q[:SOME] = ref.randn(ref.gen(51), SOME, 1, 2, D, std=1.5).to(dev)
    ws = ck.prefix_attention_workspace(q, c.k_cache, 0, TOP)
    assert ws.numel() > 16  # in parts that are joined

    def call():
        ws.fill_(0x7f)
        return ck.prefix_attention(q, c.k_cache, c.v_cache, None, 0, table, seq_lens, TOP, workspace=ws)

    def check(out):
        want, mag = c.reference(q[:SOME], D ** -0.5)
        ref.assert_attention(out[:SOME], want, mag)
        assert (out[SOME:] == 0).all()

    return call, check


def test_counts_of_parts_that_were_never_written():
    """The join behind a kernel that gave up finds counts that nobody wrote in the workspace."""
    call, check = many_empty(300_000)
    poll_ok()
    good = call()
    poll_ok()
    check(good)
    # far above any wait of the pipeline itself, below the time that 300000 lengths take to add up
    ck.set_wait_timeout_ns(20_000)
    try:
        call()
        assert ck.poll_device_status() == ck.CK_ERR_TIMEOUT
    finally:
        ck.set_wait_timeout_ns(0)
    again = call()
    poll_ok()
    assert torch.equal(again, good)


@pytest.mark.parametrize("limit", [1, 1_000, 20_000])
def test_copies_in_flight_at_a_short_limit(limit):
    """Whether a wait runs out or none does, no copy outlives its block: calls at short limits, each with its
    successor close behind, and then a right one."""
    dev = device()
    call, check = many_empty(60_000)
    g = ref.gen(52)
    q, k, v = (ref.randn(g, 2, n, 8, 128).to(dev) for n in (700, 400, 400))
    want, mag = ref.attend(q, list(k), list(v), [[400] * 700] * 2, 128 ** -0.5)
    poll_ok()
    ck.set_wait_timeout_ns(limit)
    try:
        for _ in range(10):
            call()
            ck.cross_attention(q, k, v)
        assert ck.poll_device_status() in (ck.CK_OK, ck.CK_ERR_TIMEOUT)
    finally:
        ck.set_wait_timeout_ns(0)
    ref.assert_attention(ck.cross_attention(q, k, v), want, mag)
    check(call())
    poll_ok()

"""A prompt's own attention: thousands of query tokens, each seeing the tokens up to
its own, in every way of cutting the work (fixed chunks, shares by cost, whole
groups), against the definition in 64 bits."""
import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Hq,H,page,prefix,lens", [
    (2048, 8, 2, 64, 0, [2048]),          # fixed chunks
    (8192, 8, 2, 128, 0, [8192]),         # shares by cost
    (4096, 32, 8, 64, 0, [4096]),         # whole groups, several to a CTA
    (1024, 16, 16, 16, 0, [1024] * 4),
    (1031, 6, 2, 32, 0, [1031, 1500, 2777]),
    (512, 8, 2, 64, 0, [8001]),           # a chunk behind a long history of its own
    (2100, 6, 1, 64, 700, [2100, 2300]),  # behind a shared prefix
    (1500, 4, 4, 16, 90, [1500, 400, 0, 1]),  # fewer tokens than queries: the early ones see the prefix alone
    (1500, 4, 2, 16, 0, [1500, 400, 0, 1]),   # or nothing
])
def test_prompt(Lq, Hq, H, page, prefix, lens, D):
    dev = device()
    c = ref.Paged(Lq + D, len(lens), H, D, page, prefix, lens).to(dev)
    q = ref.randn(ref.gen(Lq), len(lens), Lq, Hq, D, std=1.5).to(dev)

    def run():
        return ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, prefix, c.block_table, c.seq_lens, c.max_len)

    out = run()
    poll_ok()
    want, mag = c.reference(q, D ** -0.5)
    ref.assert_attention(out, want, mag, f"Lq{Lq} {Hq}/{H}x{D} page {page} prefix {prefix} lens {lens}")
    assert torch.equal(out, run())
    for b, n in enumerate(lens):
        if prefix == 0 and n < Lq:
            assert (out[b, :Lq - n] == 0).all()

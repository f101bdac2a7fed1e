"""The compiled calls of the 4-bit operators and the block norm: what they leave to Python to refuse, and that what
they write is theirs alone."""
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


def test_expanded_modulation_is_refused():
    """One modulation row for all groups as an expanded tensor (stride 0): refused, alone and beside rows of another
    stride; as rows of its own it is taken."""
    dev = device()
    g = ref.gen(7)
    T, H = 9, 256
    x, b = ref.randn(g, T, H).to(dev), ref.randn(g, T, H).to(dev)
    mod = ref.randn(g, 3, 3 * H, std=0.3).to(dev)
    one, own = mod[:1, :H].expand(3, H), mod[:, H:2 * H]
    q = ck._quick()
    assert q is not None, "the compiled calls were not built"
    for name in ("block_norm", "block_norm_fp4"):
        call = getattr(ck, name)
        for kw in (dict(gate=one), dict(scale=one), dict(shift=one), dict(gate=one, scale=one, shift=one), dict(gate=one, scale=own),
                   dict(gate=own, shift=one), dict(scale=one, shift=own.contiguous())):
            with pytest.raises((ValueError, ck.CkError)):
                call(x, b, tokens_per_group=4, **kw)
        got = call(x, b, tokens_per_group=4, gate=one.contiguous())
        want = call(x, b, gate=mod[:1, :H])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # the one row of a single group may be an expanded one
        got = call(x, b, tokens_per_group=T, gate=one)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    args = [x, b, None, one, 1.0, 1.0, "rms", None, None, None, None, 4, 1e-6, None, None]
    assert q.block_norm(*args) is None
    args[3], args[9] = own, one
    assert q.block_norm(*args) is None
    poll_ok()

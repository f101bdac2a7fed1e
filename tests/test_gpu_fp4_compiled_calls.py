"""The compiled calls of the 4-bit operators and the block norm: what they leave to Python to refuse, and that what
they write is theirs alone."""
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok
from test_gpu_fp4_quick_calls import H, M, Calls

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


@pytest.mark.parametrize("M", [3, 70])
def test_outputs_that_share_their_memory(M):
    """Outputs that are lazy clones: the tensors behind them keep their values, the results are those of a call with
    outputs of its own."""
    dev = device()
    g = ref.gen(M)
    H, I, fmt, t = 256, 192, "nv", 0.004
    x, b = ref.randn(g, M, H).to(dev), ref.randn(g, M, H).to(dev)
    w = ck.fp4_quantize(ref.randn(g, H, H, std=H ** -0.5).to(dev), fmt, scale=t)
    gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t)
    d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t)
    codes, scales = ck.fp4_quantize(x, fmt, scale=t)
    four = dict(x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t)
    c0, s0 = torch.full_like(codes, 0xa5), torch.full_like(scales, 0xa5)

    def row_scales(s):  # those of rows that are there
        return torch.from_numpy(ref.untile(s.cpu().numpy(), M, H, fmt))
    for given, call in [
        ((b,), lambda out=None: ck.fp4_gemm(codes, scales, *w, fmt, alpha=t * t, residual=b if out is None else out, out=out)),
        ((b,), lambda out=None: ck.fp4_linear(x, *w, fmt, x_scale=t, w_scale=t, out=out)),
        ((x,), lambda out=None: ck.fp4_linear(x if out is None else out, *w, fmt, x_scale=t, w_scale=t,
                                              residual=x if out is None else out, out=out)),
        ((x,), lambda out=None: ck.fp4_swiglu_mlp(x if out is None else out, *gu, *d, fmt, residual=x, out=out, **four)),
        ((c0, s0), lambda c=None, s=None: ck.fp4_quantize(x, fmt, scale=t, codes=c, scales=s)),
        ((x, b), lambda h=None, n=None: ck.block_norm(x, b, h_out=h, n_out=n)),
        ((x, b), lambda h=None, n=None: ck.block_norm(x if h is None else h, b if n is None else n, h_out=h, n_out=n)),
        ((x, c0, s0), lambda h=None, c=None, s=None: ck.block_norm_fp4(x, b, fmt, t, h_out=h, codes=c, scales=s)),
    ]:
        want = call()
        kept = [k.clone() for k in given]
        got = call(*[torch._lazy_clone(k) for k in given])
        for k, k0 in zip(given, kept):
            assert torch.equal(k, k0)
        want, got = (v if isinstance(v, tuple) else (v,) for v in (want, got))
        for a, e in zip(got, want):
            if a.dtype is torch.uint8 and a.dim() == 1:
                a, e = row_scales(a), row_scales(e)
            assert torch.equal(a, e)
    poll_ok()


def test_odd_columns_are_not_halved():
    dev = device()
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=dev)
    w = ck.fp4_quantize(torch.ones(16, 64, dtype=torch.bfloat16, device=dev), "nv")
    for call in (lambda x: ck.fp4_quantize(x, "nv", act="swiglu"), lambda x: ck.fp4_linear(x, *w, "nv", act="swiglu")):
        call(x[:, :128])
        with pytest.raises(ValueError):
            call(x[:, :129])
    poll_ok()


def poison(t):
    """NaN in bf16, 0xA5 in bytes: what no call here leaves."""
    t.fill_(float("nan") if t.is_floating_point() else 0xa5)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_everything_is_written_and_nothing_else(fmt):
    """Each call into poisoned outputs: given ones (and the rows' neighbours, which stay), and the memory that made
    ones will get; the Python call's results stay alive meanwhile, so that none of them is handed on."""
    c = Calls(fmt)
    assert ck._quick() is not None, "the compiled calls were not built"
    for name, args, kw in c.calls:
        given = [kw[k] for k in ("out", "h_out", "n_out", "codes", "scales") if k in kw]
        fresh = {k: torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device=v.device) if any(v is o for o in given) else v
                 for k, v in kw.items()}
        kept = getattr(ck, name)(*args, **fresh, stream=torch.cuda.current_stream())
        kept = kept if isinstance(kept, tuple) else (kept,)
        for o in given:
            poison(o if o._base is None else o._base)
        made = [torch.empty_like(k) for k in kept for _ in range(3)]
        for m in made:
            poison(m)
        del made
        got = getattr(ck, name)(*args, **kw)
        want, got = c.outputs(name, kept, fmt), c.outputs(name, got, fmt)
        for a, b in zip(got, want):
            assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b), f"{name} {list(kw)}"
        for o in given:
            if o._base is not None:  # the columns beside the rows
                beside = o._base[:, H:] if o.storage_offset() == 0 else o._base[:, :H]
                assert torch.isnan(beside).all(), name
        if "scales" in kw:  # words of rows that are not there
            rows = kw["scales"].view(-1, 32, 4, 4).permute(0, 2, 1, 3).flatten(1, 2)
            assert (rows[:, M:] == 0xa5).all(), name
    poll_ok()

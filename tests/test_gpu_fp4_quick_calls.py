"""The compiled calls of the 4-bit operators and the block norm against the same calls
through Python (a stream given takes that way): results, outputs given and made, and what
they hand back to Python to refuse."""
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

M, H, I = 9, 256, 192


class Calls:
    def __init__(self, fmt):
        dev = device()
        g = ref.gen(3)
        t = self.t = 1.0 if fmt == "mx" else 0.004
        self.x, self.branch = ref.randn(g, M, H).to(dev), ref.randn(g, M, H).to(dev)
        self.wide = ref.randn(g, M, 3 * H).to(dev)
        self.mod = ref.randn(g, 3, 3 * H, std=0.3).to(dev)
        self.w32, self.w16 = ref.randn(g, H, dtype=torch.float32).to(dev), ref.randn(g, H).to(dev)
        self.w = ck.fp4_quantize(ref.randn(g, H, H, std=H ** -0.5).to(dev), fmt, scale=t)
        self.gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t)
        self.d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t)
        codes, scales = ck.fp4_quantize(self.x, fmt, scale=t)
        x, b, w, gu, d = self.x, self.branch, self.w, self.gu, self.d
        m = dict(gate=self.mod[:, :H], scale=self.mod[:, H:2 * H], shift=self.mod[:, 2 * H:], tokens_per_group=4)
        one = dict(gate=self.mod[:1, :H], shift=self.mod[2:, 2 * H:])
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        u8 = torch.uint8
        self.calls = [
            ("fp4_quantize", (x, fmt), dict(scale=t)),
            ("fp4_quantize", (self.wide[:, H:2 * H], fmt, t), {}),
            ("fp4_quantize", (self.wide[:, :2 * H], fmt), dict(scale=t, act="swiglu")),
            ("fp4_quantize", (x.float(), fmt), dict(scale=t, codes=empty(M, H // 2, dtype=u8), scales=torch.zeros_like(scales))),
            ("fp4_gemm", (codes, scales, *w, fmt), dict(alpha=t * t)),
            ("fp4_gemm", (codes, scales, *w, fmt), dict(alpha=1, bias=self.w16, residual=b, out=empty(M, H))),
            ("fp4_linear", (x, *w, fmt), dict(x_scale=t, w_scale=t)),
            ("fp4_linear", (self.wide[:, H:], *w, fmt), dict(x_scale=t, w_scale=t, act="swiglu", bias=self.w16, residual=b,
                                                            out=empty(M, H), workspace=ck.fp4_linear_workspace(M, H, fmt))),
            ("fp4_swiglu_mlp", (x, *gu, *d, fmt), dict(x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t)),
            ("fp4_swiglu_mlp", (x, *gu, *d, fmt, t, t, t, t), dict(bgu=self.mod[0, :2 * I], bd=self.w16, residual=x, out=empty(M, H),
                                                                   workspace=ck.fp4_swiglu_mlp_workspace(M, H, I, fmt))),
            ("block_norm", (x,), {}),
            ("block_norm", (x, b), dict(weight=self.w32, bias=self.w32, post_weight=self.w32, norm="layer", eps=1e-5, **m)),
            ("block_norm", (self.wide[:, :H], self.wide[:, H:2 * H]), dict(weight=self.w16, x_factor=2, branch_factor=0.5, **one)),
            ("block_norm", (x,), dict(x_factor=0.5)),
            ("block_norm", (x, b), dict(h_out=empty(M, 2 * H)[:, :H], n_out=empty(M, 2 * H)[:, H:])),
            ("block_norm_fp4", (x, b, fmt, t), dict(weight=self.w16, norm="layer", **m)),
            ("block_norm_fp4", (x,), dict(fmt=fmt, n_scale=t, codes=empty(M, H // 2, dtype=u8), scales=torch.zeros_like(scales))),
        ]

    def outputs(self, name, got, kw):
        got = list(got) if isinstance(got, tuple) else [got]
        if name.endswith("quantize") or name == "block_norm_fp4":  # scales of rows that are not there are not written
            K = 2 * got[-2].shape[1]
            got[-1] = torch.from_numpy(ref.untile(got[-1].cpu().numpy(), M, K, kw))
        return [g.clone() for g in got]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_same_as_through_python(fmt):
    c = Calls(fmt)
    assert ck._quick() is not None, "the compiled calls were not built"
    real, used = ck._quick_module, []

    class Watch:
        def __getattr__(self, name):
            def call(*args):
                got = getattr(real, name)(*args)
                used.append(got is not None)
                return got
            return call
    for name, args, kw in c.calls:
        want = c.outputs(name, getattr(ck, name)(*args, **kw, stream=torch.cuda.current_stream()), fmt)
        torch.cuda.synchronize()
        ck._quick_module = Watch()
        try:
            got = getattr(ck, name)(*args, **kw)
        finally:
            ck._quick_module = real
        assert used.pop(), f"{name} {list(kw)}: not taken"
        given = [kw[k] for k in ("out", "h_out", "n_out", "codes", "scales") if k in kw]
        for o in given:
            assert any(o is g for g in (got if isinstance(got, tuple) else (got,))), name
        for a, b in zip(c.outputs(name, got, fmt), want):
            assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b), f"{name} {list(kw)}"
    x = c.x
    assert ck.block_norm(x)[0] is x
    poll_ok()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_what_is_not_in_order_goes_to_python(fmt):
    """None, and nothing launched: a type, a shape, strides, a device, a word, a number, a subclass, a refused size."""
    c = Calls(fmt)
    q, x, w, t = ck._quick(), c.x, c.w, c.t

    class Mine(torch.Tensor):
        pass
    ok = [x, *w, fmt, t, t, None, "none", None, None, None]
    assert q.fp4_linear(*ok) is not None
    short = w[1][:100]
    for at, bad in [(0, x.float()), (0, x.cpu()), (0, x[:, :128]), (0, x.t().contiguous().t()), (0, x[0]), (0, None), (0, 3),
                    (0, x.as_subclass(Mine)), (1, w[0].int()), (1, w[0][:, ::2]), (2, short), (3, "fp4"), (3, None), (4, "1"), (4, 0.0),
                    (5, float("nan")), (6, c.w32), (6, c.w16[:8]), (7, "gelu"), (8, x.float()), (8, x[:3]), (9, w[1][:16]),
                    (10, x[:3]), (10, c.wide[:, :H])]:
        args = list(ok)
        args[at] = bad
        if at in (4, 5) and fmt == "mx" and isinstance(bad, float):
            bad = args[at] = 0.5  # an MX tensor's scale is 1
        assert q.fp4_linear(*args) is None, (at, type(bad))
        with pytest.raises((ValueError, TypeError, AttributeError, ck.CkError, ck.ctypes.ArgumentError)):
            a = args
            ck.fp4_linear(a[0], a[1], a[2], a[3], x_scale=a[4], w_scale=a[5], bias=a[6], act=a[7], out=a[8], workspace=a[9],
                          residual=a[10]) if at != 0 or not isinstance(bad, Mine) else (_ for _ in ()).throw(ValueError)
    assert q.fp4_linear(*ok[:-1]) is None
    b = c.branch
    ok = [x, b, None, None, 1.0, 1.0, "rms", c.w16, None, None, None, 0, 1e-6, None, None]
    assert q.block_norm(*ok) is not None
    assert q.block_norm(*ok[:11], -1, *ok[12:]) is None
    # groups of more tokens than there are: one, which a row of gate is enough for
    one = list(ok)
    one[3], one[11] = b[:1], 1 << 62
    wide = q.block_norm(*one)
    one[11] = 0
    assert all(torch.equal(u, v) for u, v in zip(wide, q.block_norm(*one)))
    for at, bad in [(0, x[:, :100]), (1, b[:3]), (2, c.w32), (3, b[:0]), (3, b[:1, :8]), (4, float("inf")), (6, "batch"), (7, c.w16[:3]),
                    (8, c.w32), (9, x.float()), (11, 2.0), (11, 1 << 70), (12, -1.0), (13, x.float()), (14, x[:3])]:
        args = list(ok)
        args[at] = bad
        assert q.block_norm(*args) is None, at
    args = list(ok)
    args[3], args[11] = b[:2], 2  # five groups, two rows
    assert q.block_norm(*args) is None
    args = list(ok)
    args[3], args[10], args[11] = c.mod[:, :H], b[:3], 4  # rows at two strides
    assert q.block_norm(*args) is None
    poll_ok()

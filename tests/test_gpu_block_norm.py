"""The block norm, and the block norm to 4-bit floats, against their definition in
64 bits."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

PARTS = {
    "norm": {},
    "sum": dict(branch=1),
    "post": dict(branch=1, post_weight=1, weight=1, x_factor=0.5, branch_factor=-1.25),
    "gate": dict(branch=1, gate=1, weight=1, bias=1),
    "modulated": dict(branch=1, gate=1, scale=1, shift=1, weight=1),
    "all": dict(branch=1, post_weight=1, gate=1, scale=1, shift=1, weight=1, bias=1, x_factor=2.0, branch_factor=0.3),
    "scaled": dict(x_factor=3.0, shift=1),
}


def case(seed, T, H, parts, norm, per_group=0, wdtype=torch.bfloat16, mean=0.3):
    """Arguments of block_norm, on the CPU."""
    g = ref.gen(seed)
    a = dict(x=ref.randn(g, T, H, std=2.0, mean=mean), norm=norm, eps=1e-5, tokens_per_group=per_group)
    groups = -(-T // per_group) if per_group else 1
    p = PARTS[parts]
    if "branch" in p:
        a["branch"] = ref.randn(g, T, H, mean=-0.2)
    for name in ("post_weight", "weight", "bias"):
        if name in p:
            a[name] = ref.randn(g, H, std=0.3, mean=0.0 if name == "bias" else 1.0, dtype=wdtype)
    mod = ref.randn(g, groups, 3 * H, std=0.4)
    for i, name in enumerate(("gate", "scale", "shift")):
        if name in p:
            a[name] = mod[:, i * H:(i + 1) * H]
    for name in ("x_factor", "branch_factor"):
        if name in p:
            a[name] = p[name]
    return a


def f32_factors(a):
    return {k: float(np.float32(v)) if k.endswith("factor") or k == "eps" else v for k, v in a.items()}


def to(a, dev):
    out = {}
    mod = {n: a[n] for n in ("gate", "scale", "shift") if n in a}
    packed = None
    if mod:  # rows of one packed projection, as in use
        H = a["x"].shape[1]
        packed = torch.cat([mod.get(n, torch.zeros_like(next(iter(mod.values())))) for n in ("gate", "scale", "shift")], 1).to(dev)
    for k, v in a.items():
        if k in mod:
            i = ("gate", "scale", "shift").index(k)
            out[k] = packed[:, i * H:(i + 1) * H]
        else:
            out[k] = v.to(dev) if torch.is_tensor(v) else v
    return out


def check(a, h, n):
    want_h, want_n = ref.block_norm(**f32_factors(a))
    eh, en = ref.norm_bounds(want_h, want_n, f32_factors(a))
    for got, want, e, what in ((h, want_h, eh, "h"), (n, want_n, en, "n")):
        far = (got.double().cpu() - want).abs() - (2.0 ** -8 * (want.abs() + e) + e)
        assert float(far.max()) <= 0, f"{what}: {float(far.max())} over its bound at {int(far.argmax())}"
    poll_ok()


@pytest.mark.parametrize("parts", list(PARTS))
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,H,per", [(1, 8, 0), (5, 64, 2), (3, 264, 1), (300, 1160, 7), (37, 2048, 0), (9, 2056, 4), (21, 4096, 5),
                                     (2, 8192, 0), (7, 8200, 3), (5, 16384, 2)])
def test_block_norm(T, H, per, norm, parts):
    dev = device()
    a = case(T + H, T, H, parts, norm, per)
    check(a, *ck.block_norm(**to(a, dev)))


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_f32_weights_and_many_rows(norm):
    dev = device()
    a = case(1, 3001, 512, "all", norm, 100, wdtype=torch.float32)
    check(a, *ck.block_norm(**to(a, dev)))


@pytest.mark.parametrize("parts", ["post", "all"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,H,per", [(1311, 1480, 100), (701, 2056, 0), (607, 4096, 33), (4103, 392, 0), (9001, 264, 1000), (40001, 40, 7)])
def test_wide_threads(T, H, per, norm, parts):
    """So many rows that threads take more columns each; H fills them, or does not."""
    dev = device()
    a = case(T + H, T, H, parts, norm, per)
    check(a, *ck.block_norm(**to(a, dev)))


def test_rows_far_from_zero():
    """A mean of a thousand deviations, a channel a thousand times the others, a row of zeros, rows of tiny and huge values."""
    dev = device()
    a = case(2, 6, 1024, "sum", "layer")
    a["x"][0] += 2000
    a["x"][1, 77] = 2000
    a["x"][2], a["branch"][2] = 0, 0
    a["x"][3] *= 2.0 ** -60
    a["branch"][3] *= 2.0 ** -60
    a["x"][4] *= 2.0 ** 40
    check(a, *ck.block_norm(**to(a, dev)))
    a["norm"] = "rms"
    check(a, *ck.block_norm(**to(a, dev)))


@pytest.mark.parametrize("T,H", [(50, 576), (3, 4096)])
def test_in_place_and_rows_apart(T, H):
    dev = device()
    a = to(case(4, T, H, "all", "layer", 20), dev)
    h, n = ck.block_norm(**a)
    wide = torch.full((T, 2 * H + 16), 7.0, dtype=torch.bfloat16, device=dev)
    vx, vb = wide[:, :H], wide[:, H + 8:2 * H + 8]
    vx.copy_(a["x"]), vb.copy_(a["branch"])
    got = ck.block_norm(**{**a, "x": vx, "branch": vb}, h_out=vx, n_out=vb)
    assert got[0] is vx and got[1] is vb
    assert torch.equal(vx, h) and torch.equal(vb, n)
    assert (wide[:, H:H + 8] == 7).all() and (wide[:, 2 * H + 8:] == 7).all()
    poll_ok()


def test_stream_without_branch_is_h():
    dev = device()
    x = ref.randn(ref.gen(1), 4, 64).to(dev)
    h, n = ck.block_norm(x)
    assert h is x
    h2, n2 = ck.block_norm(x, h_out=torch.empty_like(x))
    assert torch.equal(h2, x) and torch.equal(n, n2)
    poll_ok()


def test_not_finite_stays_in_its_row():
    dev = device()
    a = case(6, 9, 320, "sum", "rms")
    a["x"][2, 5], a["branch"][4, 6] = float("nan"), float("inf")
    h, n = (t.float().cpu() for t in ck.block_norm(**to(a, dev)))
    bad = torch.zeros(9, dtype=torch.bool)
    bad[2], bad[4] = True, True
    assert torch.isnan(n[2]).all() and torch.isnan(n[4]).any()
    keep = ~bad
    a2 = {k: (v[keep] if torch.is_tensor(v) and v.shape[0] == 9 else v) for k, v in a.items()}
    check(a2, h[keep], n[keep])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,H,per,parts", [(1, 32, 0, "norm"), (5, 96, 0, "sum"), (133, 1184, 9, "all"), (40, 2080, 3, "modulated"),
                                           (1310, 1504, 9, "all"), (4103, 416, 0, "sum"), (1250, 1024, 3, "modulated"), (6, 8224, 0, "post"), (3, 16384, 2, "gate")])
def test_block_norm_fp4(T, H, per, parts, norm, fmt):
    dev = device()
    t = 1.0 if fmt == "mx" else 0.0037
    a = case(T + H, T, H, parts, norm, per)
    d = to(a, dev)
    h, codes, scales = ck.block_norm_fp4(**d, fmt=fmt, n_scale=t)
    want_h, n = ref.block_norm(**f32_factors(a))
    _, e = ref.norm_bounds(want_h, n, f32_factors(a))
    ref.assert_codes_of(ref.unpack(codes.cpu().numpy()), ref.untile(scales.cpu().numpy(), T, H, fmt), (n - e).numpy(), (n + e).numpy(),
                        fmt, t)
    assert torch.equal(h, ck.block_norm(**d)[0])
    poll_ok()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [3, 200])
def test_a_layer(T, fmt):
    """Norm, qkv-like product, MLP behind a second norm: the calls of a block in a row, as they are used, against the
    same in 64 bits on what each call was given."""
    dev = device()
    g = ref.gen(T)
    H, I = 256, 544
    t = 1.0 if fmt == "mx" else 0.004
    x, branch = ref.randn(g, T, H).to(dev), ref.randn(g, T, H).to(dev)
    w1 = ck.fp4_quantize(ref.randn(g, H, H, std=H ** -0.5).to(dev), fmt, scale=t)
    gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t)
    d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t)
    weight = ref.randn(g, H, std=0.1, mean=1.0).to(dev)
    h, codes, scales = ck.block_norm_fp4(x, branch, fmt=fmt, n_scale=t, weight=weight)
    a = ck.fp4_gemm(codes, scales, *w1, fmt, alpha=t * t)
    h2, n = ck.block_norm(h, a, weight=weight)
    y = ck.fp4_swiglu_mlp(n, *gu, *d, fmt, x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t, residual=h2)
    poll_ok()

    def val(pair, rows, K):
        return ref.values(ref.unpack(pair[0].cpu().numpy()), ref.untile(pair[1].cpu().numpy(), rows, K, fmt), fmt)
    alpha = float(np.float32(t * t))
    ref.assert_product(a, *ref.product(val((codes, scales), T, H), val(w1, H, H), alpha))
    check(dict(x=h.cpu(), branch=a.cpu(), weight=weight.cpu()), h2, n)
    hm = ck.fp4_linear(n, *gu, fmt, x_scale=t, w_scale=t)
    ref.assert_product(hm, *ref.product(val(ck.fp4_quantize(n, fmt, scale=t), T, H), val(gu, 2 * I, H), alpha))
    down = val(ck.fp4_quantize(hm, fmt, scale=t, act="swiglu"), T, I)
    ref.assert_product(y, *ref.product(down, val(d, H, I), alpha, residual=h2.double().cpu().numpy()))


def test_binding_refuses():
    dev = device()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        ck.block_norm(x, norm="batch")
    with pytest.raises(ValueError):
        ck.block_norm(x.float())
    with pytest.raises(ValueError):
        ck.block_norm(x, x[:, :32])
    with pytest.raises(ValueError):
        ck.block_norm(x, weight=torch.zeros(32, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        ck.block_norm(x, x, gate=x[:1], tokens_per_group=2)  # two groups, one row
    with pytest.raises(ck.CkError):
        ck.block_norm(x, gate=x[:1])  # no branch
    with pytest.raises(ValueError):
        ck.block_norm(x, weight=x[0], bias=x[0].float())
    with pytest.raises(ck.CkError):
        ck.block_norm_fp4(torch.zeros(4, 40, dtype=torch.bfloat16, device=dev))
    poll_ok()

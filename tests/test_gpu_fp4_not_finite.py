"""What is not finite between the two products of a SwiGLU MLP stays in its block: a weight row with a NaN scale, an
infinite bias of gate or up, an infinite or missing activation of one token."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

T = {"mx": 1.0, "nv": 0.004}
NAN_SCALE = {"mx": 255, "nv": 0x7f}
INF, NAN = float("inf"), float("nan")


def with_nan_scale(w, row, rows, K, fmt):
    """Codes and tiled scales of a weight, the scale of the row's first block a NaN."""
    codes, scales = w
    s = ref.untile(scales.cpu().numpy(), rows, K, fmt).copy()
    s[row, 0] = NAN_SCALE[fmt]
    return codes, torch.from_numpy(ref.tile(s, fmt)).to(codes.device)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [5, 20, 40, 300])
def test_weights_and_biases(M, fmt):
    """I is a multiple of 64: past 32 tokens the first product's epilogue quantizes.  What it leaves in the workspace,
    whose last part it is, against the quantizer on the first linear's result."""
    dev = device()
    g = ref.gen(M)
    H, I, t = 256, 320, T[fmt]
    x = ref.randn(g, M, H).to(dev)
    gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t)
    d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t)
    bias = ref.randn(g, 2 * I, std=0.1).to(dev)
    up_inf, gate_neg = bias.clone(), bias.clone()
    up_inf[I + 150], gate_neg[7] = INF, -INF
    gate_inf = bias.clone()
    gate_inf[319] = INF
    block = ref.BLOCK[fmt]
    for weight, b, bad in ((gu, bias, []), (with_nan_scale(gu, 37, 2 * I, H, fmt), bias, [37]),
                           (with_nan_scale(gu, I + 200, 2 * I, H, fmt), None, [200]), (gu, gate_inf, [319]), (gu, up_inf, [150]),
                           (gu, gate_neg, [7])):
        n = int(ck.lib().ck_fp4_swiglu_mlp_workspace_bytes(M, H, I, ck._FP4S[fmt]))
        ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        y = ck.fp4_swiglu_mlp(x, *weight, *d, fmt, x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t, bgu=b, workspace=ws)
        h = ck.fp4_linear(x, *weight, fmt, x_scale=t, w_scale=t, bias=b)
        want = ck.fp4_linear(h, *d, fmt, x_scale=t, w_scale=t, act="swiglu")
        poll_ok()
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
        assert torch.isnan(y).all() if bad else torch.isfinite(y).all()
        if M <= 8:
            continue  # quantized inside: no codes
        codes, scales = ck.fp4_quantize(h, fmt, scale=t, act="swiglu")
        at = n - int(ck.lib().ck_fp4_linear_workspace_bytes(M, I, ck._FP4S[fmt]))
        got_codes = ref.unpack(ws[at:at + M * I // 2].view(M, I // 2).cpu().numpy())
        at += -(-(M * I // 2) // 256) * 256
        got_scales = ref.untile(ws[at:at + scales.numel()].cpu().numpy(), M, I, fmt)
        want_scales = ref.untile(scales.cpu().numpy(), M, I, fmt)
        assert np.array_equal(got_scales, want_scales)
        nan = got_scales == NAN_SCALE[fmt]
        assert sorted(set(np.argwhere(nan)[:, 1])) == [c // block for c in bad]
        assert not bad or nan[:, bad[0] // block].all()
        same = ref.unpack(codes.cpu().numpy()) == got_codes
        assert (same | np.repeat(nan, block, axis=1)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [5, 20, 70])
def test_one_token(M, fmt):
    """The second linear on [gate | up] of which one token has an infinity and one a NaN: these rows are NaN, the
    others as they are beside finite ones."""
    dev = device()
    g = ref.gen(M + 1)
    N, I, t = 64, 192, T[fmt]
    w = ck.fp4_quantize(ref.randn(g, N, I, std=I ** -0.5).to(dev), fmt, scale=t)
    h = ref.randn(g, M, 2 * I).to(dev)
    kw = dict(x_scale=t, w_scale=t, act="swiglu")
    plain = ck.fp4_linear(h, *w, fmt, **kw)
    h[2, 17], h[4, I + 100] = INF, NAN
    y = ck.fp4_linear(h, *w, fmt, **kw)
    poll_ok()
    rows = torch.zeros(M, dtype=torch.bool, device=dev)
    rows[[2, 4]] = True
    assert torch.isnan(y[rows]).all() and torch.equal(y[~rows], plain[~rows])

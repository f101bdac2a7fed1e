"""The example's decoder layer on 4-bit weights: norms, projections, attention and MLP together."""
import os
import sys

import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("B,prompt,steps,with_states", [(1, 16, 1, False), (4, 150, 5, True), (12, 33, 20, True), (40, 20, 2, False)])
def test_decoder_layer(B, prompt, steps, with_states, fmt):
    device()
    import decoder_layer
    error, y = decoder_layer.run(B, prompt, steps, with_states, fmt=fmt)
    # bf16 output and bf16 probabilities: 2^-8 each at most, both far less over a row
    assert error <= 2.0 ** -7
    assert y.shape[0] == B and torch.isfinite(y.float()).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("B", [3, 70])
def test_mlp_behind_its_norm(B, fmt):
    """The end of a layer against the same calls of the library one by one."""
    dev = device()
    import decoder_layer
    layer = decoder_layer.Fp4DecoderLayer(fmt, device=dev)
    g = ref.gen(B)
    x, branch = ref.randn(g, B, 512).to(dev), ref.randn(g, B, 512).to(dev)
    y = layer._mlp(x, branch, layer.out)
    o, gu, d = layer.out, layer.gate_up, layer.down
    a = ck.fp4_gemm(*ck.fp4_quantize(branch, fmt, scale=o.x_scale), o.W, o.scales, fmt, alpha=o.x_scale * o.scale)
    h, n = ck.block_norm(x, a, weight=layer.norm_mlp)
    gate_up = ck.fp4_linear(n, gu.W, gu.scales, fmt, x_scale=gu.x_scale, w_scale=gu.scale)
    want = ck.fp4_linear(gate_up, d.W, d.scales, fmt, x_scale=d.x_scale, w_scale=d.scale, act="swiglu", residual=h)
    poll_ok()
    assert torch.equal(y, want)

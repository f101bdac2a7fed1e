"""The example's decoder layer: projections, append, rotation, attention and MLP
together, a batch behind a shared prompt."""
import os
import sys

import pytest
import torch

from gpu_helpers import device

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,prompt,steps,with_states", [(1, 16, 1, False), (4, 150, 5, True), (12, 33, 20, True)])
def test_decoder_layer(B, prompt, steps, with_states):
    device()
    import decoder_layer
    error, y = decoder_layer.run(B, prompt, steps, with_states)
    # bf16 output and bf16 probabilities: 2^-8 each at most, both far less over a row
    assert error <= 2.0 ** -7
    assert y.shape[0] == B and torch.isfinite(y.float()).all()

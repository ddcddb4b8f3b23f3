"""The example layer: trained by the operators' gradients, then served in 8 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_layer_learns_and_serves():
    got = example().main(steps=60)
    assert got["last"] < 0.8 * got["first"]
    # two 8-bit products in a row, each value off by at most half of 1/127 of its row's largest
    # (about 4 standard deviations here): some 1% of the norm each; 5% is ample
    assert got["error"] < 0.05


def test_layer_without_tokens_and_with_one():
    layer = example().ExpertLayer(64, 96, 4, 2)
    for tokens in (0, 1):
        x = torch.randn(tokens, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        out = layer(x)
        assert out.shape == (tokens, 64) and out.dtype == torch.bfloat16
        out.float().sum().backward()
        assert x.grad.shape == x.shape and layer.up.grad.isfinite().all()

"""Gradients of the expert-layer operators where a graph of them is asked for."""
from __future__ import annotations

import pytest
import torch

from test_experts_gpu import layer, layer_inputs, normal

pytestmark = pytest.mark.gpu


def test_first_order_with_and_without_a_graph():
    leaves, ids, num = layer_inputs()
    out = layer(leaves[0], ids, *leaves[1:], num)
    seed = normal(9, *out.shape, dtype=out.dtype)
    want = torch.autograd.grad(out, leaves, seed, retain_graph=True)
    for a, b in zip(torch.autograd.grad(out, leaves, seed, create_graph=True), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("first", range(4))
def test_second_order_is_refused(first):
    leaves, ids, num = layer_inputs()
    out = layer(leaves[0], ids, *leaves[1:], num)
    grad, = torch.autograd.grad(out.float().sum(), leaves[first], create_graph=True)
    with pytest.raises(RuntimeError, match="first order"):
        (grad.float().square().sum() + out.float().sum()).backward()

"""Gradients of the expert-layer operators where a graph of them is asked for."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import groups, layer, layer_inputs, normal, route

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


def test_merge_without_weights():
    g = groups(route(1, 30, 3, 4), 4)
    y = normal(2, 90, 72, dtype=torch.bfloat16).requires_grad_()
    out = experts.merge(y, g, None)
    assert torch.equal(out, experts.combine(y.detach(), g))
    seed = normal(3, *out.shape, dtype=out.dtype)
    grad, = torch.autograd.grad(out, y, seed)
    want = torch.where(g.order.view(-1, 1) >= 0, seed[g.order.long().clamp(min=0) // 3], 0)
    assert torch.equal(grad, want)

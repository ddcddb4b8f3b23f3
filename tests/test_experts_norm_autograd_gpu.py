"""Where the gradient that h gets from what follows is added to the norm's."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,n", [(1, 8), (33, 300), (70, 2048)])
def test_the_gradient_of_h(rows, n, dtype):
    """With a residual within the norm's backward pass; without one h is x, and the sum is autograd's."""
    x, residual = normal(1, rows, n, dtype=dtype), normal(2, rows, n, dtype=dtype)
    weight = (1 + 0.2 * normal(3, n)).to(dtype)
    by_y, by_h = normal(4, rows, n, dtype=dtype), normal(5, rows, n, dtype=dtype)
    leaves = [t.clone().requires_grad_() for t in (x, weight, residual)]
    y, h = experts.norm(*leaves)
    dx, dweight, dresidual = torch.autograd.grad((y, h), leaves, (by_y, by_h))
    want, want_weight = experts.rms_norm_backward(by_y, h.detach(), weight, by_h)
    assert torch.equal(dx, want) and torch.equal(dresidual, want) and torch.equal(dweight, want_weight)
    y, h = experts.norm(*leaves[:2])
    assert h is leaves[0]
    dx, dweight = torch.autograd.grad((y, h), leaves[:2], (by_y, by_h))
    rounded, want_weight = experts.rms_norm_backward(by_y, x, weight)
    assert torch.equal(dx, rounded + by_h) and torch.equal(dweight, want_weight)

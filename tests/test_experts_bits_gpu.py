"""A product's bits do not depend on its operands' addresses: views with padded rows, off 16 bytes,
take other tiles and other loops than contiguous ones."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import int8_weight, normal
from test_experts_kernels_gpu import ROWS, WEIGHTS, names, pairs_of

pytestmark = pytest.mark.gpu


def shifted(t, by):
    """The same values, each row `by` elements into a longer one."""
    longer = torch.zeros(*t.shape[:-1], t.shape[-1] + 2 * by + 3, dtype=t.dtype, device=t.device)
    view = longer[..., by:by + t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("size", [c[1] for c in ROWS], ids=names(ROWS))
@pytest.mark.parametrize("by", [1, 4])
def test_products_of_rows(size, by):
    tokens, num, n, k = size
    g = pairs_of(tokens, num)
    x, w = normal(1, tokens, k, dtype=torch.bfloat16), normal(2, num, n, k, dtype=torch.bfloat16)
    assert torch.equal(experts.matmul(shifted(x, by), shifted(w, by), g, gather=True),
                       experts.matmul(x, w, g, gather=True))
    dy, w = normal(3, tokens, k, dtype=torch.float16), normal(4, num, k, n, dtype=torch.float16)
    assert torch.equal(experts.matmul_dx(shifted(dy, by), shifted(w, by), g),
                       experts.matmul_dx(dy, w, g))
    xq, sx = experts.quantize_rows(x)
    wq, sw = int8_weight(5, num, n, k)
    assert torch.equal(experts.int8_matmul(shifted(xq, by), sx, shifted(wq, by), sw, g, gather=True),
                       experts.int8_matmul(xq, sx, wq, sw, g, gather=True))


@pytest.mark.parametrize("size", [c[1] for c in WEIGHTS], ids=names(WEIGHTS))
@pytest.mark.parametrize("by", [1, 4])
def test_gradient_of_the_weights(size, by):
    tokens, num, n, k = size
    g = pairs_of(tokens, num)
    x, dy = normal(1, tokens, k, dtype=torch.bfloat16), normal(2, tokens, n, dtype=torch.bfloat16)
    assert torch.equal(experts.matmul_dw(shifted(dy, by), shifted(x, by), g, gather=True),
                       experts.matmul_dw(dy, x, g, gather=True))

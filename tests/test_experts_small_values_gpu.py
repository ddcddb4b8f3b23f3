"""Operands and results below the smallest normal number of their type (tolerances as in
test_experts_gpu; a 32-bit sum below its own smallest normal number is off by half a step of 2^-149 for each
addition besides)."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import assert_close, groups, normal, product, route, spans

pytestmark = pytest.mark.gpu

# thin, 32 x 128, 64 x 64, 128 x 128 and 256 x 256 straight to LDS, and through registers
SIZES = [(12, 6, 64, 64), (160, 8, 4000, 96), (200, 2, 2600, 136), (1000, 8, 4008, 136),
         (4100, 1, 4104, 520), (1500, 2, 5601, 137)]


def subnormal(seed, *shape, dtype):
    """Whole multiples of the smallest number, up to the smallest normal one."""
    info = torch.finfo(dtype)
    steps = (normal(seed, *shape).abs() * 0.3 / info.eps).round().clamp(1, 1 / info.eps - 1)
    sign = torch.where(normal(seed + 1, *shape) < 0, -1.0, 1.0)
    value = (steps * sign).double() * (info.smallest_normal * info.eps)
    out = value.to(dtype)
    assert torch.equal(out.double(), value) and float(out.abs().max()) < info.smallest_normal
    return out


@pytest.mark.parametrize("tokens,num,n,k", SIZES)
@pytest.mark.parametrize("dtype,scale", [(torch.float16, 512.0), (torch.bfloat16, 2.0**30)])
def test_subnormal_operands(tokens, num, n, k, dtype, scale):
    """Each operand in turn, the other so large that the products are normal numbers."""
    g = groups(route(tokens, tokens, 1, num, "all"), num)
    small, large = subnormal(1, tokens, k, dtype=dtype), normal(3, num, n, k, dtype=dtype) * scale
    y = experts.matmul(small, large, g)
    dy = normal(5, tokens, n, dtype=dtype) * scale
    tiny = subnormal(6, num, n, k, dtype=dtype)
    dw, dx = experts.matmul_dw(dy, small, g), experts.matmul_dx(dy, tiny, g)
    for e, a, b in spans(g):
        assert_close(y[a:b], *product(small[a:b], large[e]), k)
        assert_close(dw[e], *product(dy[a:b].t(), small[a:b].t()), max(1, b - a))
        assert_close(dx[a:b], *product(dy[a:b], tiny[e].t()), n)


@pytest.mark.parametrize("tokens,num,n,k", SIZES)
def test_subnormal_results(tokens, num, n, k):
    """float16 results below 2^-14, from normal operands."""
    g = groups(route(tokens, tokens, 1, num, "all"), num)
    x = normal(1, tokens, k, dtype=torch.float16, scale=2.0**-9)
    w = normal(2, num, n, k, dtype=torch.float16, scale=2.0**-9 * k**-0.5)
    y = experts.matmul(x, w, g)
    assert float(y.abs().max()) < 2.0**-14
    for e, a, b in spans(g):
        assert_close(y[a:b], *product(x[a:b], w[e]), k)


def test_subnormal_rows_combine():
    g = groups(route(1, 40, 3, 5), 5)
    for dtype in (torch.float16, torch.bfloat16):
        y = subnormal(1, 120, 136, dtype=dtype)
        weights = normal(2, 40, 3)
        has = (g.place >= 0).unsqueeze(2)
        rows = torch.where(has, y.double()[g.place.long().clamp(min=0)], 0.0)
        each = rows * weights.double().unsqueeze(2)
        assert_close(experts.combine(y, g, weights), each.sum(1),
                     each.abs().sum(1) + 2.0**-126, 4)

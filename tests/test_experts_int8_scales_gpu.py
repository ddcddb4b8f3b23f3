"""The 8-bit product's scaling and sums at the ends of their ranges (tolerances as in
test_experts_gpu)."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import assert_int8, groups, int8_weight, normal, route, spans, token_rows

pytestmark = pytest.mark.gpu

# rows, columns, reduction: divided among waves; 64 x 64 and 128 x 128 straight to LDS; through registers
DENSE = [(1, 500, 1024), (40, 300, 2048), (200, 2600, 1168), (1000, 4008, 1152), (200, 2603, 397)]


@pytest.mark.parametrize("rows,n,k", DENSE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("large", [1e33, 3e38])
def test_large_rows_with_small_weights(rows, n, k, dtype, large):
    """What a row's scale and the whole-number sum make together may not be finite, as long as the
    result is."""
    x = normal(1, rows, k).clamp(-4, 4) * (large / 4)
    xq, sx = experts.quantize_rows(x.bfloat16())
    assert sx.isfinite().all()
    wq, sw = int8_weight(2, n, k)
    sw = sw / large
    y = experts.int8_matmul(xq, sx, wq, sw, out_dtype=dtype)
    assert y.isfinite().all()
    sums = xq.double() @ wq.double().t().contiguous()
    assert_int8(y, sums, sx.view(-1, 1), sw.view(1, -1))


@pytest.mark.parametrize("tokens,num,n,k", [(30, 6, 500, 1024), (600, 5, 4008, 1152)])
def test_large_rows_by_expert(tokens, num, n, k):
    g = groups(route(tokens, tokens, 2, num), num)
    size = 10.0**(normal(2, tokens, 1) * 12)
    size[::5] = 1e37
    x = (normal(1, tokens, k) * size.clamp(1e-30, 1e37)).bfloat16()
    xq, sx = experts.quantize_rows(x)
    wq, sw = int8_weight(3, num, n, k)
    sw = sw * 1e-6
    y = experts.int8_matmul(xq, sx, wq, sw, g, gather=True)
    for e, a, b in spans(g):
        sums = token_rows(xq, g, a, b, True).double() @ wq[e].double().t().contiguous()
        assert_int8(y[a:b], sums, token_rows(sx, g, a, b, True).view(-1, 1), sw[e].view(1, -1))


@pytest.mark.parametrize("rows,n", [(1, 20), (300, 4100)])
def test_scales_that_are_zero_subnormal_or_not_finite(rows, n):
    k = 64
    xq = torch.ones(rows, k, dtype=torch.int8, device="cuda")
    wq = torch.ones(n, k, dtype=torch.int8, device="cuda")
    wq[:, 1::2] = -1
    wq[5] = 1
    sw = torch.full((n,), 0.5, device="cuda")
    sw[0], sw[1], sw[2], sw[3] = 0.0, float("inf"), float("nan"), 2.0**-149
    sw[4] = -2.0
    for scale in (0.0, 2.0**-149, 1.0, 2.0**127, float("inf"), float("nan")):
        sx = torch.full((rows,), scale, device="cuda")
        y = experts.int8_matmul(xq, sx, wq, sw)
        sums = (xq.double() @ wq.double().t().contiguous())
        want = (sums * sx.double().view(-1, 1) * sw.double()).bfloat16()
        assert torch.equal(y.isnan(), want.isnan())
        ok = ~want.isnan()
        assert torch.equal(y[ok], want[ok])


@pytest.mark.parametrize("rows,n", [(1, 20), (40, 300), (300, 4100)])
def test_the_largest_sums_of_the_widest_reduction(rows, n):
    """k = 131072: -128 throughout sums to 2^31, -128 times 127 to its opposite less 2^24."""
    k = 2**17
    xq = torch.full((rows, k), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    wq[2, 5] = -127
    wq[3, k // 2:] = 127
    one = torch.ones(max(rows, n), device="cuda")
    y = experts.int8_matmul(xq, one[:rows], wq, one[:n])
    sums = xq[:1].double() @ wq.double().t().contiguous()
    assert int(sums[0, 0]) == 2**31
    assert_int8(y, sums.expand(rows, n), one[:rows].view(-1, 1), one[:n].view(1, -1))

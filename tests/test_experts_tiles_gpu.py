"""Every kernel that a product can take, by sizes that lead to it, with ragged ends in rows,
columns and reduction, against the products in 64 bits (tolerances as in test_experts_gpu)."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import (assert_close, assert_int8, groups, int8_weight, normal, product,
                              route, spans, token_rows)

pytestmark = pytest.mark.gpu

# (tokens, experts, columns of the result, reduction); one choice a token
SIZES = [
    (4100, 1, 4200, 136),   # 256 x 256, its last round divided
    (5000, 9, 4104, 264),   # 256 x 256 over ragged groups
    (1600, 16, 8200, 200),  # 128 x 256
    (1000, 8, 4008, 144),   # 128 x 128
    (1000, 8, 2000, 1160),  # 128 x 128, four stages
    (480, 8, 4000, 328),    # 64 x 128
    (160, 8, 4008, 264),    # 32 x 128, short reduction
    (160, 8, 4000, 1096),   # 32 x 128
    (200, 2, 2600, 1160),   # 64 x 64
    (30, 2, 500, 1032),     # 32 x 64, the reduction divided among waves
    (12, 6, 500, 1032),     # 16 x 16, likewise
    (1500, 2, 5601, 137),   # 256 x 128 through registers
    (1000, 8, 4001, 335),   # 128 x 128 through registers
    (200, 2, 2603, 397),    # 64 x 64, or 32 x 128, through registers
    (300, 3, 100, 331),     # fewer columns than a tile, through registers
]


def pairs_of(tokens, num):
    return groups(route(tokens, tokens, 1, num), num)


@pytest.mark.parametrize("tokens,num,n,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matmul(tokens, num, n, k, dtype):
    g = pairs_of(tokens, num)
    x, w = normal(1, tokens, k, dtype=dtype), normal(2, num, n, k, dtype=dtype, scale=k**-0.5)
    y = experts.matmul(x, w, g, gather=True)
    assert (y[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        assert_close(y[a:b], *product(token_rows(x, g, a, b, True), w[e]), k)


@pytest.mark.parametrize("tokens,num,n,k", SIZES)
@pytest.mark.parametrize("aligned", [False, True])
def test_int8(tokens, num, n, k, aligned):
    k = (k + 15) // 16 * 16 if aligned else k  # 16-byte rows: straight to LDS
    g = pairs_of(tokens, num)
    xq, sx = experts.quantize_rows(normal(1, tokens, k, dtype=torch.bfloat16))
    wq, sw = int8_weight(2, num, n, k)
    y = experts.int8_matmul(xq, sx, wq, sw, g, gather=True)
    assert (y[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        sums = token_rows(xq, g, a, b, True).double() @ wq[e].double().t().contiguous()
        assert_int8(y[a:b], sums, token_rows(sx, g, a, b, True).view(-1, 1), sw[e].view(1, -1))


@pytest.mark.parametrize("tokens,num,k,n", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matmul_dx(tokens, num, k, n, dtype):
    g = pairs_of(tokens, num)
    dy, w = normal(1, tokens, n, dtype=dtype), normal(2, num, n, k, dtype=dtype, scale=n**-0.5)
    dx = experts.matmul_dx(dy, w, g)
    assert (dx[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        assert_close(dx[a:b], *product(dy[a:b], w[e].t()), n)


@pytest.mark.parametrize("tokens,num,n,k", [
    (300, 2, 2600, 2104),   # 256 x 256
    (1000, 70, 520, 264),   # 256 x 256, more experts than lanes
    (700, 300, 264, 144),   # more experts than 256, most with few rows
    (500, 3, 264, 392),     # 128 x 128
    (300, 2, 2601, 3003),   # 256 x 128 through registers
    (500, 3, 265, 393),     # 128 x 128 through registers
    (400, 2, 77, 333),      # fewer rows of the weight than a tile
])
@pytest.mark.parametrize("gather", [True, False])
def test_matmul_dw(tokens, num, n, k, gather):
    g = pairs_of(tokens, num)
    x = normal(1, tokens, k, dtype=torch.bfloat16)
    dy = normal(2, tokens, n, dtype=torch.bfloat16, scale=(tokens / num)**-0.5)
    dw = experts.matmul_dw(dy, x, g, gather=gather)
    for e, a, b in spans(g):
        assert_close(dw[e], *product(dy[a:b].t(), token_rows(x, g, a, b, gather).t()),
                     max(1, b - a))


@pytest.mark.parametrize("n,k", [(4104, 200), (4100, 205)])
def test_values_that_are_not_finite_stay_in_large_tiles(n, k):
    """A row, a column or an expert with an infinity leaves the others' bits."""
    g = pairs_of(5000, 4)
    x, w = normal(1, 5000, k, dtype=torch.float16), normal(2, 4, n, k, dtype=torch.float16)
    y = experts.matmul(x, w, g)
    kept = int(g.offsets[-1])
    x[257, k - 1] = float("inf")
    w[1, n - 1, k - 1] = float("nan")
    got = experts.matmul(x, w, g)
    fine = torch.ones_like(y, dtype=torch.bool)
    fine[257] = False
    fine[int(g.offsets[1]):int(g.offsets[2]), n - 1] = False
    assert torch.equal(got[fine], y[fine]) and (got[kept:] == 0).all()
    assert not got[257].isfinite().any()
    assert got[int(g.offsets[1]):int(g.offsets[2]), n - 1].isnan().all()

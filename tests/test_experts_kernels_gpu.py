"""Every kernel of the products in the loops that its sizes let it take: whole steps and ragged ends,
last rounds that are divided, waves without rows (tolerances as in test_experts_gpu). That each size
reaches the kernel that it names is checked without a GPU by test_experts_kernels_cpu."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import (assert_close, assert_int8, groups, int8_weight, normal, product,
                              route, spans, token_rows)

pytestmark = pytest.mark.gpu

# kernel: (rows, columns, stages, straight to LDS). What the products of rows take for (tokens, experts,
# columns of the result, reduction in 16-bit elements); one choice a token. The gradient of the rows has
# its own kernel where it is given.
LARGE, WIDE, ALONE, SQUARE = (256, 256, 2, 1), (128, 256, 3, 1), (128, 128, 4, 1), (128, 128, 2, 1)
ROWS = [
    ("large, last round divided", (4100, 1, 4104, 520), LARGE, None),
    ("large, ragged groups", (5000, 9, 4104, 648), LARGE, None),
    ("large, in one round", (2800, 16, 2696, 584), LARGE, None),
    ("128 x 256", (1600, 16, 8200, 520), WIDE, None),
    ("128 x 128, one on a CU", (1000, 8, 2000, 1160), ALONE, None),
    ("128 x 128", (1000, 8, 4008, 520), SQUARE, None),
    ("128 x 128, short", (3000, 4, 2504, 328), SQUARE, None),
    ("64 x 128", (480, 8, 4000, 1032), (64, 128, 3, 1), None),
    ("32 x 128, short", (160, 8, 4008, 264), (32, 128, 2, 1), None),
    ("32 x 128", (160, 8, 4000, 1096), (32, 128, 4, 1), (32, 128, 3, 1)),
    ("64 x 64", (200, 2, 2600, 1160), (64, 64, 3, 1), (64, 128, 3, 1)),
    ("32 x 64, divided reduction", (30, 2, 500, 1160), (32, 64, 0, 0), None),
    ("16 x 16, divided reduction", (12, 6, 500, 4232), (16, 16, 0, 0), None),
]
# through registers: reductions off 16 bytes
VIA = [
    ("256 x 128", (1500, 2, 5601, 777), (256, 128, 2, 0), None),
    ("128 x 128", (1000, 8, 4001, 777), (128, 128, 2, 0), None),
    ("64 x 64", (200, 2, 2603, 781), (64, 64, 2, 0), (32, 128, 2, 0)),
]
# the gradient of the weights: (tokens, experts, rows and columns of the weight)
WEIGHTS = [
    ("256 x 256", (1300, 2, 2600, 2104), LARGE),
    ("256 x 256, many experts", (4001, 24, 1016, 1016), LARGE),
    ("128 x 128", (2400, 3, 264, 392), SQUARE),
    ("256 x 128 through registers", (1700, 2, 2601, 2043), (256, 128, 2, 0)),
    ("128 x 128 through registers", (2400, 3, 265, 393), (128, 128, 2, 0)),
]


def names(cases):
    return [c[0].replace(" ", "_") for c in cases]


def by_rows(f):
    return pytest.mark.parametrize("size", [c[1] for c in ROWS + VIA], ids=names(ROWS) + [
        n + "_through_registers" for n in names(VIA)])(f)


def pairs_of(tokens, num):
    """One expert takes all tokens; several take what a router gives them, and some are dropped."""
    return groups(route(tokens, tokens, 1, num, "all" if num == 1 else "mixed"), num)


def test_the_large_cases_are_what_they_say():
    """Row tiles of 256 as the kernels count them."""
    tokens, num, n, _ = ROWS[0][1]
    high = (pairs_of(tokens, num).counts.long() + 255) // 256
    last = int(high.sum()) * ((n + 255) // 256) % 256
    assert 0 < last <= 128  # divided
    assert 0 < tokens % 256 <= 128  # and a tile with waves that have no rows
    ragged = pairs_of(*ROWS[1][1][:2]).counts
    assert (ragged % 256 != 0).any() and (ragged > 256).any()


@by_rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matmul(size, dtype):
    tokens, num, n, k = size
    g = pairs_of(tokens, num)
    x, w = normal(1, tokens, k, dtype=dtype), normal(2, num, n, k, dtype=dtype, scale=k**-0.5)
    y = experts.matmul(x, w, g, gather=True)
    assert (y[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        assert_close(y[a:b], *product(token_rows(x, g, a, b, True), w[e]), k)


@by_rows
def test_int8(size):
    tokens, num, n, k = size
    k = 2 * k  # as many bytes
    if size in [c[1] for c in VIA]:
        k += 1
    g = pairs_of(tokens, num)
    xq, sx = experts.quantize_rows(normal(1, tokens, k, dtype=torch.bfloat16))
    wq, sw = int8_weight(2, num, n, k)
    y = experts.int8_matmul(xq, sx, wq, sw, g, gather=True)
    assert (y[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        sums = token_rows(xq, g, a, b, True).double() @ wq[e].double().t().contiguous()
        assert_int8(y[a:b], sums, token_rows(sx, g, a, b, True).view(-1, 1), sw[e].view(1, -1))


@by_rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matmul_dx(size, dtype):
    tokens, num, k, n = size
    g = pairs_of(tokens, num)
    dy, w = normal(1, tokens, n, dtype=dtype), normal(2, num, n, k, dtype=dtype, scale=n**-0.5)
    dx = experts.matmul_dx(dy, w, g)
    assert (dx[int(g.offsets[-1]):] == 0).all()
    for e, a, b in spans(g):
        assert_close(dx[a:b], *product(dy[a:b], w[e].t()), n)


@pytest.mark.parametrize("size", [c[1] for c in WEIGHTS], ids=names(WEIGHTS))
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matmul_dw(size, gather, dtype):
    tokens, num, n, k = size
    g = pairs_of(tokens, num)
    x = normal(1, tokens, k, dtype=dtype)
    dy = normal(2, tokens, n, dtype=dtype, scale=(tokens / num)**-0.5)
    dw = experts.matmul_dw(dy, x, g, gather=gather)
    for e, a, b in spans(g):
        assert_close(dw[e], *product(dy[a:b].t(), token_rows(x, g, a, b, gather).t()),
                     max(1, b - a))


@pytest.mark.parametrize("num", [1, 9])
def test_values_that_are_not_finite_stay_in_the_large_kernels(num):
    """A row or a column with an infinity leaves the others' bits, forward and back."""
    tokens, _, n, k = ROWS[0][1] if num == 1 else ROWS[1][1]
    g = pairs_of(tokens, num)
    last = int(g.offsets[-1]) - 1
    x, w = normal(1, tokens, k, dtype=torch.float16), normal(2, num, n, k, dtype=torch.float16)
    y = experts.matmul(x, w, g)
    x[last, k - 1] = float("inf")
    w[0, n - 1, k - 1] = float("nan")
    got = experts.matmul(x, w, g)
    fine = torch.ones_like(y, dtype=torch.bool)
    fine[last] = False
    fine[:int(g.offsets[1]), n - 1] = False
    assert torch.equal(got[fine], y[fine])
    assert not got[last].isfinite().any() and got[:int(g.offsets[1]), n - 1].isnan().all()
    # (columns of the result and reduction change places, as in test_matmul_dx)
    dy, w = normal(3, tokens, k, dtype=torch.float16), normal(4, num, k, n, dtype=torch.float16)
    dx = experts.matmul_dx(dy, w, g)
    dy[last, k - 1] = float("nan")
    w[0, k - 1, n - 1] = float("inf")
    got = experts.matmul_dx(dy, w, g)
    assert torch.equal(got[fine], dx[fine])
    assert not got[last].isfinite().any()
    assert not got[:int(g.offsets[1]), n - 1].isfinite().any()

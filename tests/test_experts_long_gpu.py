"""More rows than one launch takes (2^32 - 1 threads): the documented limit is 2^30."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import assert_close, quantized

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def random(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def straight(tokens, top_k):
    """Every pair in its own place, apart from a dropped one near each end."""
    pairs = tokens * top_k
    place = torch.arange(pairs, dtype=torch.int32, device="cuda")
    for i in (3, pairs - 2):
        place[i] = -1
    order = place.clone()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    return experts.Groups(none, torch.zeros(2, dtype=torch.int32, device="cuda"), order,
                          place.view(tokens, top_k))


def test_combine():
    tokens, n = 2**28 + 5, 8  # 16 lanes a token
    g = straight(tokens, 1)
    y = random(1, tokens, n)
    out = experts.combine(y, g)
    y[3], y[tokens - 2] = 0, 0
    assert torch.equal(out, y)
    weights = torch.full((tokens, 1), 2.0, device="cuda")
    weights[-1] = 0.5
    y *= 2
    y[-1] *= 0.25  # 0.5 in all
    assert torch.equal(experts.combine(out, g, weights), y)


def test_combine_backward():
    tokens, top_k, n = 2**25 + 3, 2, 8  # a wave a pair
    g = straight(tokens, top_k)
    dout, y = random(1, tokens, n), random(2, tokens * top_k, n)
    weights = random(3, tokens, top_k, dtype=torch.float32)
    dy, dweights = experts.combine_backward(dout, y, g, weights)
    kept = (g.place >= 0).view(-1, 1)
    rows = dout.float().repeat_interleave(top_k, 0)
    assert torch.equal(dy, torch.where(kept, weights.view(-1, 1) * rows, 0.0).bfloat16())
    products = torch.where(kept, rows * y.float(), 0.0)  # exact: 16 bits of digits
    assert_close(dweights.view(-1), products.double().sum(1), products.abs().double().sum(1), n)


def test_quantize_narrow_rows():
    rows, k = 2**26 + 7, 8  # a wave a row
    x = random(1, rows, k)
    x[5], x[-2] = 0, 0
    xq, sx = experts.quantize_rows(x)
    for a in range(0, rows, 2**24):
        q, scale = quantized(x[a:a + 2**24])
        assert torch.equal(sx[a:a + 2**24].double(), scale)
        assert torch.equal(xq[a:a + 2**24].double(), q)


def test_quantize_wide_rows():
    rows, k = 2**24 + 3, 1032  # a workgroup a row
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 2**23, 2**24 - 2, 2**24 - 1, 2**24, rows - 1], device="cuda")
    x[some] = random(1, some.numel(), k)
    xq, sx = experts.quantize_rows(x)
    q, scale = quantized(x[some])
    assert torch.equal(xq[some].double(), q) and torch.equal(sx[some].double(), scale)
    assert int(torch.count_nonzero(sx)) == some.numel()
    xq[some] = 0
    assert all(int(xq[a:a + 2**21].amax()) == 0 == int(xq[a:a + 2**21].amin())
               for a in range(0, rows, 2**21))

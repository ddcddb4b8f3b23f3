"""The norm, its 8-bit form and its gradients against their formulas in 64 bits.

Tolerances, from the arithmetic alone: a result is rounded once to its type (half a step, finfo.eps / 2
of the value, or half the smallest subnormal). A lane of at least 64 adds at most ceil(n / 512) * 8 terms
one after another, a wave's 64 lanes are added in 6 steps and 16 waves in 16, so that a 32-bit sum over a
row is off by at most chain(n) = n / 64 + 8 + 22 times 2^-24 of the sum of its terms' magnitudes (each step
rounds by 2^-24). Ten more roundings cover the mean, the root, the reciprocal and the products that follow.
"""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import normal

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
# a wave, a workgroup and the largest one a row; ragged and odd widths; rows past registers
WIDTHS = [1, 2, 7, 8, 63, 512, 515, 1024, 1500, 2048, 2056, 4095, 4096, 5000, 8192, 8200, 16384, 16391,
          32768, 40003]
U = 2.0**-24


def chain(n):
    return n / 64 + 30


def formula(x, weight, residual, eps):
    """(y, h) in 64 bits; h as it is stored."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = h.double()
    return d / (d.square().mean(1, keepdim=True) + eps).sqrt() * weight.double(), h


def half_step(want, dtype):
    info = torch.finfo(dtype)
    return want.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def assert_within(got, want, room):
    bad = ~((got.double() - want).abs() <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], room[bad][:4])


def inputs(seed, rows, n, dtype, residual, scale=1.0):
    x = normal(seed, rows, n, dtype=dtype, scale=scale)
    weight = (1 + 0.2 * normal(seed + 1, n)).to(dtype)
    return x, weight, normal(seed + 2, rows, n, dtype=dtype, scale=3 * scale) if residual else None


def check_norm(x, weight, residual, eps=1e-5):
    n = x.shape[1]
    want, h = formula(x, weight, residual, eps)
    y, got_h = experts.rms_norm(x, weight, residual, eps)
    assert y.dtype == x.dtype and torch.equal(got_h, h)
    assert got_h is x or residual is not None
    # (the sum's error counts half in its root)
    assert_within(y, want, half_step(want, x.dtype) * 1.01 + want.abs() * ((chain(n) / 2 + 10) * U))
    xq, sx, got_h = experts.rms_norm_int8(x, weight, residual, eps)
    assert xq.shape == x.shape and xq.stride(0) % 16 == 0 and torch.equal(got_h, h)
    top = want.abs().amax(1)
    relative = (chain(n) / 2 + 12) * U
    assert_within(sx, top / 127, top / 127 * relative + 2.0**-149)
    steps = torch.where(top > 0, 127 / top, 0.0).view(-1, 1) * want
    assert_within(xq, steps, 0.5 + 127 * 2 * relative + torch.zeros_like(steps))


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(n, dtype, residual):
    for rows in (1, 5, 70):
        check_norm(*inputs(rows * n, rows, n, dtype, residual))


def gradients(dy, h, weight, dh, eps):
    """dx, dweight in 64 bits, and the magnitudes of what their sums add."""
    n = h.shape[1]
    d, g, w = h.double(), dy.double(), weight.double()
    r = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    u, dn = d * r, g * w
    along = (dn * u).mean(1, keepdim=True)
    dx = r * (dn - u * along)
    size = r * (dn.abs() + u.abs() * (dn * u).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    assert n == dx.shape[1]
    return dx, size, (g * u).sum(0), (g * u).abs().sum(0)


def check_gradients(dy, h, weight, dh, eps=1e-5):
    rows, n = h.shape
    dx, dweight = experts.rms_norm_backward(dy, h, weight, dh, eps)
    want, size, want_w, size_w = gradients(dy, h, weight, dh, eps)
    # (r enters dx as its third power at most, and along has a sum of its own)
    assert_within(dx, want, half_step(want, dy.dtype) * 1.01 + size * ((2.5 * chain(n) + 20) * U))
    # the groups add rows / groups terms each; then 32 lanes add groups / 32 and 5 more
    terms = rows + 64 + 6
    assert_within(dweight, want_w, half_step(want_w, dy.dtype) * 1.01 +
                  size_w * ((chain(n) / 2 + 10 + terms) * U))
    return dx, dweight


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_gradients(n, dtype, with_dh):
    for rows in (1, 6, 67):
        h, weight, dh = inputs(rows * n, rows, n, dtype, with_dh)
        check_gradients(normal(rows * n + 3, rows, n, dtype=dtype), h, weight, dh)


@pytest.mark.parametrize("rows,n", [(9001, 500), (5003, 1000), (3001, 2048), (2500, 4096), (700, 8192),
                                    (600, 16384), (200, 17000)])
def test_many_rows(rows, n):
    """More rows than groups of them, so that each group has several."""
    dtype = torch.bfloat16
    x, weight, residual = inputs(n, rows, n, dtype, True)
    check_norm(x, weight, residual)
    check_gradients(normal(n + 3, rows, n, dtype=dtype), x, weight, residual)


@pytest.mark.parametrize("n", [100, 2000, 9000, 40000])
def test_views(n):
    """Padded rows off 16 bytes: the same bits, and nothing around them is touched."""
    x, weight, residual = inputs(n, 20, n, torch.bfloat16, True)
    dy = normal(n + 5, 20, n, dtype=torch.bfloat16)

    def shifted(t):
        longer = torch.full((20, n + 11), float("nan"), dtype=t.dtype, device="cuda")
        longer[:, 3:3 + n] = t
        return longer[:, 3:3 + n]

    for a, b in zip(experts.rms_norm(shifted(x), weight, shifted(residual)),
                    experts.rms_norm(x, weight, residual)):
        assert torch.equal(a, b)
    for a, b in zip(experts.rms_norm_int8(shifted(x), weight, shifted(residual)),
                    experts.rms_norm_int8(x, weight, residual)):
        assert torch.equal(a, b)
    for a, b in zip(experts.rms_norm_backward(shifted(dy), shifted(x), weight, shifted(residual)),
                    experts.rms_norm_backward(dy, x, weight, residual)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [64, 3000, 20000])
def test_large_values(n):
    """Rows whose squares pass the range of 32 bits, beside ordinary ones and rows of zeros."""
    x, weight, _ = inputs(n, 6, n, torch.bfloat16, False)
    x[1] *= 1e30
    x[2] = 3e38
    x[3] = 0
    x[4, 5:] = 0
    x[4, :5] = 1e25
    check_norm(x, weight, None)
    dy = normal(n + 3, 6, n, dtype=torch.bfloat16)
    check_gradients(dy, x, weight, None)
    dx, _ = experts.rms_norm_backward(dy, x, weight)
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("n", [64, 3000, 20000])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_row(n, value):
    x, weight, residual = inputs(n, 5, n, torch.float16, True)
    x[2, n // 2] = value
    y, h = experts.rms_norm(x, weight, residual)
    fine = [0, 1, 3, 4]
    want, _ = formula(x, weight, residual, 1e-6)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.isnan(y[2, n // 2])
    clean = x.clone()
    clean[2] = 0
    assert torch.equal(y[fine], experts.rms_norm(clean, weight, residual)[0][fine])
    xq, sx, _ = experts.rms_norm_int8(x, weight, residual)
    assert torch.isnan(sx[2]) and not xq[2].any() and torch.isfinite(sx[fine]).all()
    dx, dweight = experts.rms_norm_backward(residual, x, weight)
    assert torch.isnan(dx[2]).any() and torch.isfinite(dx[fine]).all()


def test_small_weights_and_scales():
    """Scales without a normal reciprocal."""
    x, _, _ = inputs(1, 4, 256, torch.bfloat16, False)
    weight = torch.full((256,), 1e-38, dtype=torch.bfloat16, device="cuda")
    xq, sx, _ = experts.rms_norm_int8(x, weight)
    want, _ = formula(x, weight, None, 1e-6)
    # the scale is subnormal: half a step of 2^-149 of a scale near 3e-40 moves a quotient by at most
    # 127 * 2^-150 / scale, and y itself as much
    room = 0.5 + 127 * 2.0**-148 / (want.abs().amax(1) / 127).view(-1, 1) + 1e-3
    assert_within(xq, want / (want.abs().amax(1) / 127).view(-1, 1), room + torch.zeros_like(want))
    zero = experts.rms_norm_int8(x, torch.zeros_like(weight))
    assert not zero[0].any() and not zero[1].any()


def test_no_rows():
    x = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    weight = torch.ones(48, dtype=torch.bfloat16, device="cuda")
    assert experts.rms_norm(x, weight, x)[0].shape == (0, 48)
    assert experts.rms_norm_int8(x, weight)[0].shape == (0, 48)
    dx, dweight = experts.rms_norm_backward(x, x, weight)
    assert dx.shape == (0, 48) and dweight.shape == (48,) and not dweight.any()


def test_refused():
    x, weight, residual = inputs(1, 4, 64, torch.bfloat16, True)
    for bad in (lambda: experts.rms_norm(x, weight.half()), lambda: experts.rms_norm(x, weight[:8]),
                lambda: experts.rms_norm(x, weight, residual[:3]),
                lambda: experts.rms_norm(x, weight, residual.half()),
                lambda: experts.rms_norm(x, weight, residual.cpu()),
                lambda: experts.rms_norm(x, weight, eps=0.0),
                lambda: experts.rms_norm(x[:, ::2], weight[:32]),
                lambda: experts.rms_norm(x[0], weight),
                lambda: experts.rms_norm_backward(x, residual[:2], weight),
                lambda: experts.rms_norm_backward(x, residual, weight, x.half())):
        with pytest.raises(ValueError):
            bad()


def test_autograd_and_differences():
    """The gradients that autograd takes, against differences of the formula in 64 bits along a
    direction; x and the residual get the same gradient."""
    dtype = torch.float16
    x, weight, residual = inputs(7, 33, 300, dtype, True)
    leaves = [t.clone().requires_grad_() for t in (x, weight, residual)]
    y, h = experts.norm(*leaves, eps=1e-5)
    by_y, by_h = normal(8, 33, 300, dtype=dtype), normal(9, 33, 300, dtype=dtype)
    grads = torch.autograd.grad((y, h), leaves, (by_y, by_h))
    assert torch.equal(grads[0], grads[2])
    want, size, want_w, size_w = gradients(by_y, h.detach(), weight, by_h, 1e-5)
    assert_within(grads[0], want, half_step(want, dtype) * 1.01 + size * ((2.5 * chain(300) + 20) * U))

    def value(h, weight):
        y = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * weight
        return (y * by_y.double()).sum() + (h * by_h.double()).sum()

    at = [h.detach().double(), weight.double()]
    step = [torch.randn_like(t) for t in at]
    delta = 1e-6
    difference = (value(*[a + delta * s for a, s in zip(at, step)]) -
                  value(*[a - delta * s for a, s in zip(at, step)])) / (2 * delta)
    along = sum((g.double() * s).sum() for g, s in zip((grads[0], grads[1]), step))
    # each gradient is off by half a step of its value, at random signs at worst all alike
    room = sum((half_step(g.double(), dtype) * 1.1 * s.abs()).sum()
               for g, s in zip((grads[0], grads[1]), step)) + difference.abs() * 1e-6
    assert (along - difference).abs() <= room
    only_h, = torch.autograd.grad(experts.norm(*leaves)[1], leaves[0], by_h)
    assert torch.equal(only_h, by_h)


def test_captured_twice_and_on_another_stream():
    x, weight, residual = inputs(1, 700, 2048, torch.bfloat16, True)
    dy = normal(5, 700, 2048, dtype=torch.bfloat16)

    def run():
        y, h = experts.rms_norm(x, weight, residual)
        return (y, h, *experts.rms_norm_int8(y, weight, h)[:2],
                *experts.rms_norm_backward(dy, h, weight, y))

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    captured = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        captured.append((graph, out))
    stream = torch.cuda.Stream()
    for _ in range(3):
        for graph, out in captured:
            for t in out:
                t.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            again = run()
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))

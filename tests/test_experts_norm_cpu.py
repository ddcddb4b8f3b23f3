"""The norm without a GPU: refusals, workspace sizes, and what autograd makes of it with the kernels
replaced by formulas in 64 bits."""
from __future__ import annotations

import ctypes

import pytest
import torch

from partitioned_chip_accumulation_amd import experts, hist
from test_experts_cpu import BAD, OK, UNSUPPORTED, P, calls

NAN, INF = float("nan"), float("inf")


def test_argument_errors_before_any_device_call():
    bad_eps = [(11, 0.0), (11, -1.0), (11, NAN), (11, INF), (11, 1e-31)]
    good = (P, 64, P, 64, P, 64, P, 64, P, 10, 64, 1e-6, 0)
    calls("experts_rms_norm", good,
          [(0, None), (0, P + 1), (1, 63), (2, None), (3, 63), (4, None), (5, 63), (6, P + 1), (7, 63),
           (8, None), (8, P + 1), (10, 0), (12, 2), (12, -1)] + bad_eps)
    calls("experts_rms_norm_int8", (P, 64, P, P, 64, P, 64, P, 64, P, 10, 64, 1e-6, 0),
          [(0, None), (1, 63), (2, None), (2, P + 2), (3, None), (4, 63), (5, None), (6, 63),
           (8, 63), (9, None), (11, 0), (12, 0.0), (13, 2)])
    lib = experts._library()
    for change in ((9, 2**30 + 1), (10, 2**17 + 1)):
        args = list(good)
        args[1] = args[3] = args[5] = args[7] = 2**18
        args[change[0]] = change[1]
        assert lib.experts_rms_norm(*args, None) == UNSUPPORTED

    back = (P, 64, P, P, 64, P, 64, P, 64, P, 10, 64, 1e-6, 0, P, 2**20)
    calls("experts_rms_norm_backward", back,
          [(0, None), (1, 63), (2, None), (2, P + 1), (3, None), (4, 63), (5, None), (6, 63), (7, P + 1),
           (8, 63), (9, None), (11, 0), (12, 0.0), (13, 2)])
    for ws, size in ((None, 2**20), (P + 8, 2**20), (P, 2559)):
        args = back[:14] + (ws, size)
        assert lib.experts_rms_norm_backward(*args, None) == hist.HIST_ERR_WORKSPACE


def test_workspace_size():
    size = experts._library().experts_rms_norm_backward_workspace_size
    n = ctypes.c_uint64(0)
    assert size(10, 64, ctypes.byref(n)) == OK and n.value == 10 * 64 * 4
    assert size(0, 64, ctypes.byref(n)) == OK and n.value == 0
    assert size(2**30, 2**17, ctypes.byref(n)) == OK and n.value < 2**33
    assert size(10, 0, ctypes.byref(n)) == BAD and size(10, 64, None) == BAD
    assert size(2**30 + 1, 64, ctypes.byref(n)) == UNSUPPORTED
    assert size(10, 2**17 + 1, ctypes.byref(n)) == UNSUPPORTED


def test_tensors_of_the_host_are_refused():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for call in (lambda: experts.rms_norm(x, x[0]), lambda: experts.rms_norm_int8(x, x[0], x),
                 lambda: experts.rms_norm_backward(x, x, x[0]), lambda: experts.norm(x, x[0])):
        with pytest.raises(ValueError):
            call()


def plain(x, weight, residual=None, eps=1e-6):
    h = x if residual is None else x + residual
    return h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * weight, h


def plain_backward(dy, h, weight, dh=None, eps=1e-6):
    r = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    dn = dy * weight
    dx = r * (dn - h * r * r * (dn * h).mean(1, keepdim=True))
    return dx if dh is None else dx + dh, (dy * h * r).sum(0)


@pytest.fixture
def opaque(monkeypatch):
    """The module's calls, computed on the host, without a graph."""
    def replace(name, fn):
        def call(*args, **kwargs):
            with torch.no_grad():
                return fn(*args, **kwargs)
        monkeypatch.setattr(experts, name, call)

    replace("rms_norm", plain)
    replace("rms_norm_backward", plain_backward)


def leaves(residual):
    gen = torch.Generator().manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64).requires_grad_()

    return [normal(6, 10), normal(10)] + ([normal(6, 10)] if residual else [])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_gradients_are_those_of_the_formula(opaque, residual, use):
    inputs = leaves(residual)

    def loss(fn):
        y, h = fn(*inputs, eps=1e-3)
        return (y.sin().sum() if use != "h" else 0) + (h.cos().sum() if use != "y" else 0)

    got = torch.autograd.grad(loss(experts.norm), inputs, allow_unused=True)
    want = torch.autograd.grad(loss(plain), inputs, allow_unused=True)
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        if a is not None:
            torch.testing.assert_close(a, b, rtol=1e-12, atol=1e-12)


def test_gradients_against_differences(opaque):
    inputs = leaves(True)
    weigh = [torch.randn(6, 10, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
             for i in (1, 2)]
    assert torch.autograd.gradcheck(
        lambda *a: sum((o * w).sum() for o, w in zip(experts.norm(*a, eps=1e-3), weigh)), inputs)


@pytest.mark.parametrize("residual", [False, True])
def test_shared_and_broadcast_leaves(opaque, residual):
    """x that is its own residual, and rows that are one row expanded."""
    x, weight, *_ = leaves(False)
    row = x[:1].detach().requires_grad_()

    def loss(fn):
        rows = row.expand(6, 10)
        y, h = fn(x + rows, weight, x if residual else None)
        return (y * y.cos()).sum() + h.sin().sum()

    got = torch.autograd.grad(loss(experts.norm), (x, row, weight))
    want = torch.autograd.grad(loss(plain), (x, row, weight))
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("first", range(3))
def test_a_gradient_of_a_gradient_is_refused(opaque, first):
    inputs = leaves(True)
    y, h = experts.norm(*inputs)
    grad, = torch.autograd.grad(y.square().sum() + h.sum(), inputs[first], create_graph=True)
    with pytest.raises(RuntimeError, match="first order"):
        (grad.square().sum() + y.sum()).backward()

"""What autograd makes of the expert-layer operators, without a GPU: the kernels' calls are replaced
by plain products in 64 bits that, like the kernels, leave no graph behind them."""
from __future__ import annotations

import pytest
import torch

from partitioned_chip_accumulation_amd import experts

TOKENS, TOP_K, NUM, N, K = 7, 2, 3, 5, 4


def tokens_of(x, g, gather):
    return x[g.order.long() // g.place.shape[1]] if gather else x


def expert_of(g):
    return torch.repeat_interleave(torch.arange(g.counts.numel()), g.counts.long())


def plain_matmul(x, w, g, gather=False):
    return torch.einsum("pk,pnk->pn", tokens_of(x, g, gather), w[expert_of(g)])


def plain_combine(y, g, weights=None):
    rows = y[g.place.long()]
    return (rows if weights is None else rows * weights.unsqueeze(2)).sum(1)


def plain_dx(dy, w, g):
    return torch.einsum("pn,pnk->pk", dy, w[expert_of(g)])


def plain_dw(dy, x, g, gather=False):
    each = torch.einsum("pn,pk->pnk", dy, tokens_of(x, g, gather))
    return torch.zeros(NUM, N, x.shape[1], dtype=x.dtype).index_add(0, expert_of(g), each)


def plain_combine_backward(dout, y, g, weights):
    t = g.order.long() // g.place.shape[1]
    dy = dout[t] * weights.reshape(-1)[g.order.long()].unsqueeze(1)
    return dy, (dout.unsqueeze(1) * y[g.place.long()]).sum(2)


@pytest.fixture
def opaque(monkeypatch):
    """The module's calls, computed on the host, without a graph."""
    def replace(name, fn):
        def call(*args, **kwargs):
            with torch.no_grad():
                return fn(*args, **kwargs)
        monkeypatch.setattr(experts, name, call)

    replace("matmul", plain_matmul)
    replace("matmul_dx", plain_dx)
    replace("matmul_dw", plain_dw)
    replace("combine", plain_combine)
    replace("combine_backward", plain_combine_backward)


def inputs():
    gen = torch.Generator().manual_seed(3)
    ids = torch.rand(TOKENS, NUM, generator=gen).topk(TOP_K, dim=1).indices
    key = ids.reshape(-1)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel())
    counts = torch.bincount(key, minlength=NUM)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    g = experts.Groups(*[t.int() for t in (counts, offsets, order, place.view_as(ids))])

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64).requires_grad_()

    return g, normal(TOKENS, K), normal(NUM, N, K), normal(TOKENS, TOP_K)


def layer(linear, merge, g, x, w, weights):
    return merge(torch.tanh(linear(x, w, g, gather=True)), g, weights)


def test_first_gradients_are_those_of_the_formula(opaque):
    g, *leaves = inputs()
    out = layer(experts.linear, experts.merge, g, *leaves)
    want = layer(plain_matmul, plain_combine, g, *leaves)
    torch.testing.assert_close(out, want, rtol=1e-12, atol=1e-12)
    wants = torch.autograd.grad(want.square().sum(), leaves)
    for create_graph in (False, True):
        got = torch.autograd.grad(out.square().sum(), leaves, retain_graph=True,
                                  create_graph=create_graph)
        for a, b in zip(got, wants):
            torch.testing.assert_close(a, b, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("first", range(3))
def test_a_gradient_of_a_gradient_is_refused(opaque, first):
    """A penalty on a gradient of the layer beside a term that autograd can differentiate: what the
    gradient's own kernels add must not be left out."""
    g, *leaves = inputs()
    out = layer(experts.linear, experts.merge, g, *leaves)
    grad, = torch.autograd.grad(out.square().sum(), leaves[first], create_graph=True)
    with pytest.raises(RuntimeError, match="first order"):
        (grad.square().sum() + out.sum()).backward()


def test_refused_too_where_the_gradient_that_comes_in_is_a_constant(opaque):
    g, x, w, weights = inputs()
    for out, leaf in ((experts.linear(x, w, g, gather=True), x),
                      (experts.linear(x, w, g, gather=True), w),
                      (experts.merge(experts.linear(x, w, g, gather=True), g, weights), weights)):
        grad, = torch.autograd.grad(out.sum(), leaf, create_graph=True)
        assert grad.requires_grad
        with pytest.raises(RuntimeError, match="first order"):
            (grad.square().sum() + x.sum() + w.sum() + weights.sum()).backward()
    y = plain_matmul(x, w, g, True).detach().requires_grad_()
    grad, = torch.autograd.grad(experts.merge(y, g, weights).sum(), y, create_graph=True)
    with pytest.raises(RuntimeError, match="first order"):
        (grad.square().sum() + weights.sum()).backward()


def test_a_gradient_that_depends_on_no_leaf_stays_a_constant(opaque):
    g, x, w, weights = inputs()
    fixed = w.detach()
    grad, = torch.autograd.grad(experts.linear(x, fixed, g, gather=True).sum(), x,
                                create_graph=True)
    assert not grad.requires_grad
    y = plain_matmul(x, w, g, True).detach().requires_grad_()
    grad, = torch.autograd.grad(experts.merge(y, g, weights.detach()).sum(), y, create_graph=True)
    assert not grad.requires_grad


def test_merge_without_weights_adds_the_rows(opaque):
    """As combine does without weights; the rows' gradients are the tokens'."""
    g, x, w, _ = inputs()
    y = plain_matmul(x, w, g, True).detach().requires_grad_()
    out = experts.merge(y, g, None)
    want = plain_combine(y, g)
    torch.testing.assert_close(out, want, rtol=1e-12, atol=1e-12)
    seed = torch.randn(*out.shape, dtype=out.dtype)
    for a, b in zip(torch.autograd.grad(out, y, seed), torch.autograd.grad(want, y, seed)):
        torch.testing.assert_close(a, b, rtol=1e-12, atol=1e-12)

"""A mixture-of-experts layer with partitioned_chip_accumulation_amd.experts.

Trains a small layer on synthetic data (group, grouped products, weighted sum and their
gradients), then answers single tokens and a batch with its weights in 8 and in 4 bits.

    python examples/expert_layer.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from partitioned_chip_accumulation_amd import experts  # noqa: E402


class ExpertLayer(torch.nn.Module):
    """top_k of num experts, each down(silu(up(x))), for bfloat16 or float16 rows."""

    def __init__(self, width, hidden, num, top_k, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.num, self.top_k = num, top_k

        def weight(*shape):
            w = torch.randn(*shape, device=device) * shape[-1]**-0.5
            return torch.nn.Parameter(w.to(dtype))

        self.router = torch.nn.Parameter(torch.randn(width, num, device=device) * width**-0.5)
        self.up, self.down = weight(num, hidden, width), weight(num, width, hidden)

    def route(self, x):
        score, ids = (x.float() @ self.router).topk(self.top_k, dim=1)
        return ids, score.softmax(dim=1)

    def forward(self, x):
        ids, weights = self.route(x)
        g = experts.group_rows(ids, self.num)
        h = torch.nn.functional.silu(experts.linear(x, self.up, g, gather=True))
        return experts.merge(experts.linear(h, self.down, g), g, weights)


class Int8ExpertLayer:
    """The same layer for serving: weights in 8 bits with a scale for each output channel. A few tokens
    go through it in one call, their rows in 16 bits; more of them through grouped 8-bit products."""
    quantize = staticmethod(experts.quantize_rows)
    product = staticmethod(experts.int8_matmul)

    def __init__(self, layer: ExpertLayer):
        self.route, self.num = layer.route, layer.num
        self.up, self.down = (self._quantized(w.detach()) for w in (layer.up, layer.down))

    @classmethod
    def _quantized(cls, w):
        q, scale = cls.quantize(w.reshape(-1, w.shape[2]))
        return q.reshape(*w.shape[:2], -1).contiguous(), scale.view(w.shape[:2])

    @torch.no_grad()
    def __call__(self, x):
        ids, weights = self.route(x)
        if x.shape[0] <= experts.MAX_FEW:
            return experts.few_tokens(x, self.up, self.down, ids, weights, gated=False)
        g = experts.group_rows(ids, self.num)
        h = self.product(*self.quantize(x), *self.up, g, gather=True, out_dtype=x.dtype)
        h = torch.nn.functional.silu(h)
        y = self.product(*self.quantize(h), *self.down, g, out_dtype=x.dtype)
        return experts.combine(y, g, weights)


class Mx4ExpertLayer(Int8ExpertLayer):
    """Weights in 4 bits with a power of two for each block of 32."""
    quantize = staticmethod(experts.quantize_mx4)
    product = staticmethod(experts.mx4_matmul)

    @classmethod
    def _quantized(cls, w):
        q, powers = cls.quantize(w.reshape(-1, w.shape[2]))
        return q.view(*w.shape[:2], -1), powers.view(*w.shape[:2], -1)


def main(steps: int = 100, width: int = 256, hidden: int = 512, num: int = 16, top_k: int = 2,
         tokens: int = 2048) -> dict:
    torch.manual_seed(0)
    layer = ExpertLayer(width, hidden, num, top_k)
    target = torch.randn(width, width, device="cuda") * width**-0.5
    optimizer = torch.optim.Adam(layer.parameters(), lr=1e-3)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16)
        loss = (layer(x).float() - torch.tanh(x.float() @ target)).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if step % 20 == 0 or step == steps - 1:
            print(f"step {step:4d}  loss {losses[-1]:.4f}", flush=True)

    x = torch.randn(64, width, device="cuda", dtype=torch.bfloat16)
    many = x.repeat(4, 1)
    with torch.no_grad():
        want = layer(x).float()
    found = {}
    for name, served in (("8", Int8ExpertLayer(layer)), ("4", Mx4ExpertLayer(layer))):
        singles = torch.cat([served(x[i:i + 1]) for i in range(x.shape[0])]).float()
        batch = served(many)[:x.shape[0]].float()
        found[name] = [float((got - want).norm() / want.norm()) for got in (singles, batch)]
        print(f"in {name} bits: relative difference of single tokens {found[name][0]:.4f}, "
              f"of a batch {found[name][1]:.4f}")
    return {"first": float(losses[0]), "last": float(losses[-1]), "error": found["8"][0],
            "batch": found["8"][1], "mx4": found["4"][0], "mx4_batch": found["4"][1]}


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=100)
    main(parser.parse_args().steps)

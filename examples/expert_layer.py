"""A mixture-of-experts layer with partitioned_chip_accumulation_amd.experts.

Trains a small layer on synthetic data (group, grouped products, weighted sum and their
gradients), then answers single tokens with its weights in 8 bits.

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
        return experts.group_rows(ids, self.num), score.softmax(dim=1)

    def forward(self, x):
        g, weights = self.route(x)
        h = torch.nn.functional.silu(experts.linear(x, self.up, g, gather=True))
        return experts.merge(experts.linear(h, self.down, g), g, weights)


class Int8ExpertLayer:
    """The same layer for serving: weights in 8 bits with a scale for each output channel."""

    def __init__(self, layer: ExpertLayer):
        self.route = layer.route
        self.up, self.down = (self._quantized(w.detach()) for w in (layer.up, layer.down))

    @staticmethod
    def _quantized(w):
        q, scale = experts.quantize_rows(w.reshape(-1, w.shape[2]))
        return q.reshape(w.shape).contiguous(), scale.view(w.shape[:2])

    @torch.no_grad()
    def __call__(self, x):
        g, weights = self.route(x)
        h = experts.int8_matmul(*experts.quantize_rows(x), *self.up, g, gather=True,
                                out_dtype=x.dtype)
        h = torch.nn.functional.silu(h)
        y = experts.int8_matmul(*experts.quantize_rows(h), *self.down, g, out_dtype=x.dtype)
        return experts.combine(y, g, weights)


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

    served = Int8ExpertLayer(layer)
    x = torch.randn(64, width, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        want = layer(x).float()
    got = torch.cat([served(x[i:i + 1]) for i in range(x.shape[0])]).float()
    error = float((got - want).norm() / want.norm())
    print(f"single tokens in 8 bits: relative difference {error:.4f}")
    return {"first": float(losses[0]), "last": float(losses[-1]), "error": error}


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=100)
    main(parser.parse_args().steps)

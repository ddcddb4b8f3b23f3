"""The expert layer's lines in README.md run as they stand."""
from __future__ import annotations

import os
import re

import pytest
import torch

from partitioned_chip_accumulation_amd import experts
from test_experts_gpu import normal

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_lines_run():
    with open(os.path.join(ROOT, "README.md")) as f:
        code, = re.findall(r"```python\n(from partitioned_chip_accumulation_amd import experts\n.*?)```",
                           f.read(), re.S)
    num, width, hidden, tokens = 6, 96, 64, 20
    bf16 = torch.bfloat16
    w_up = normal(1, num, hidden, width, dtype=bf16)
    wq, sw = experts.quantize_rows(w_up.view(-1, width))
    wc, wp = experts.quantize_mx4(w_up.view(-1, width))
    names = dict(
        torch=torch, num_experts=num, x=normal(2, tokens, width, dtype=bf16), w_up=w_up,
        w_down=normal(3, num, width, hidden, dtype=bf16), weights=normal(4, tokens, 2).softmax(1),
        ids=torch.stack([torch.arange(tokens) % num, (torch.arange(tokens) + 1) % num], 1).int().cuda(),
        wq=wq.view(num, hidden, width), sw=sw.view(num, hidden),
        wc=wc.view(num, hidden, -1), wp=wp.reshape(num, hidden, -1),
        weight=normal(5, width, dtype=bf16), residual=normal(6, tokens, width, dtype=bf16))
    exec(code, names)
    assert names["out"].shape == (tokens, width) and torch.isfinite(names["out"]).all()
    assert names["h"].shape == (2 * tokens, hidden)

"""The 8-bit norm rounds y / sx as it says, to the nearest whole number with ties to even.

Rows of 1 and -1 have a norm of 1 (eps is far below the last bit of 1), so y is the weight and nothing in it is
rounded: what each value becomes is known exactly. sx is max / 127 rounded to 32 bits, and a value times 2 and an
odd number of up to 8 bits times sx are exact in 64 bits, so comparing them decides."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from partitioned_chip_accumulation_amd import experts

pytestmark = pytest.mark.gpu


def nearest(a, scale):
    """a / scale for a >= 0 to the nearest whole number, ties to even."""
    m = np.floor(a / scale)
    twice, middle = 2 * a, (2 * m + 1) * scale
    return np.where(twice == middle, m + m % 2, m + (twice > middle))


# a top value of 1.125 makes 0.5625 lie next to 63.5 steps; 40 of the 128 tops of bfloat16 have such a value
@pytest.mark.parametrize("bits,dtype", [(7, torch.bfloat16), (10, torch.float16)])
@pytest.mark.parametrize("power", [0, -100])
def test_every_value_below_a_largest_one(bits, dtype, power):
    """All values of eight binades below each of the largest ones (every fifth one of float16's)."""
    if dtype == torch.float16:
        power = power // 20  # (within its range)
    binade = 1 + np.arange(2**bits) / 2.0**bits
    every = np.concatenate([binade * 2.0**-e for e in range(8)])
    wrong = []
    for top in binade[::5 if bits == 10 else 1]:
        value = every[every <= top] * 2.0**power
        weight = torch.from_numpy(value * np.where(np.arange(value.size) % 3 == 0, -1.0, 1.0)).to(dtype).cuda()
        x = torch.ones(2, value.size, dtype=dtype, device="cuda")
        x[1, ::2] = -1
        xq, sx, _ = experts.rms_norm_int8(x, weight, eps=1e-30)
        scale = float(np.float32(top * 2.0**power) / np.float32(127))
        assert (sx.double().cpu().numpy() == scale).all()
        want = nearest(value, scale)
        got = (xq.double() * x.double() * torch.sign(weight.double())).cpu().numpy()
        wrong += [(top, v, g, w) for row in got for v, g, w in zip(value, row, want) if g != w]
    assert not wrong, (len(wrong), wrong[:5])

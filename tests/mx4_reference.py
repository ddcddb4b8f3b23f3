"""The 4-bit form of rows, written from its definition in numpy, for the tests of the operators on it."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks_of(x):
    """[rows, blocks, 32] in 64 bits, zeros past the end."""
    x = np.asarray(x, dtype=np.float64)
    more = -x.shape[1] % 32
    return np.pad(x, ((0, 0), (0, more))).reshape(x.shape[0], -1, 32)


def codes_of(a):
    """The codes of values that are divided by their power: nearest, ties to the even code, at most 6."""
    size = np.abs(a)
    code = np.zeros(a.shape, dtype=np.uint8)
    for c in range(1, 8):
        middle = (GRID[c - 1] + GRID[c]) / 2
        code = np.where(size >= middle if c % 2 == 0 else size > middle, c, code)
    return (code + 8 * np.signbit(a)).astype(np.uint8)


def quantize(x):
    """(codes [rows, 16 blocks], powers [rows, blocks])"""
    blocks = blocks_of(x)
    with np.errstate(invalid="ignore"):
        top = np.abs(blocks).max(axis=2)
    finite = np.isfinite(top)
    exponent = np.frexp(np.where(finite, top, 1.0))[1] - 1
    power = np.where(top == 0, -127, np.clip(exponent - 2, -127, 127)).astype(np.int64)
    scaled = np.where(finite[..., None], np.ldexp(blocks, -power[..., None].astype(np.int32)), 0.0)
    code = codes_of(scaled)
    code = np.where(finite[..., None], code, 0).reshape(x.shape[0], -1)
    # (past the row's end the padding is +0)
    return ((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8),
            np.where(finite, power + 127, 255).astype(np.uint8))


def values(codes, powers):
    """What codes and powers of any leading dimensions stand for, in 64 bits."""
    codes, powers = np.asarray(codes), np.asarray(powers)
    code = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1, 32)
    size = np.where(code >= 8, -GRID[code & 7], GRID[code & 7])
    scale = np.where(powers == 255, np.nan, np.ldexp(1.0, powers.astype(np.int32) - 127))
    return (size * scale[..., None]).reshape(*codes.shape[:-1], -1)

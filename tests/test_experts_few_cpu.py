"""The layer for a few tokens without a GPU: refusals and workspace sizes."""
from __future__ import annotations

import ctypes

import pytest
import torch

from partitioned_chip_accumulation_amd import experts, hist
from test_experts_cpu import BAD, OK, UNSUPPORTED, P


def weight(kind=0, ld=128, stride=8192, scales=None, ld_scales=0, scales_stride=0, data=P):
    return experts._Weight(data, ld, stride, scales, ld_scales, scales_stride, kind)


def call(change=(), up=None, down=None):
    up = weight() if up is None else up
    down = weight(ld=64) if down is None else down
    args = [P, 96, P, 128, ctypes.addressof(up), ctypes.addressof(down), P, 32, P, 10, 2, 4, 128, 64,
            96, 1, 0, P, 2**24, None]
    for at, value in change:
        args[at] = value
    return experts._library().experts_few_tokens(*args)


def test_argument_errors_before_any_device_call():
    for at, value in [(0, None), (0, P + 1), (1, 95), (2, None), (2, P + 1), (3, 127), (4, None),
                      (5, None), (6, None), (6, P + 2), (7, 16), (8, None), (8, P + 2), (10, 0), (11, 0),
                      (12, 0), (13, 0), (14, 0), (15, 2), (15, -1), (16, 2), (16, -1)]:
        assert call([(at, value)]) == BAD, (at, value)
    for at, value in [(9, 65), (10, 65), (11, 1025), (12, 2**17 + 1), (13, 2**17 + 1), (14, 2**17 + 1),
                      (9, 2**63)]:
        big = weight(ld=2**18)
        change = [(at, value), (1, 2**18), (3, 2**18)]
        assert call(change, big, weight(ld=2**18)) == UNSUPPORTED, (at, value)
    for ws, size in ((None, 2**24), (P + 8, 2**24), (P, 64)):
        assert call([(17, ws), (18, size)]) == hist.HIST_ERR_WORKSPACE
    for bad in (weight(kind=3), weight(kind=-1), weight(ld=127), weight(stride=-1),
                weight(data=None), weight(data=P + 1), weight(kind=1),
                weight(kind=1, scales=P + 2), weight(kind=1, scales=P, scales_stride=-1),
                weight(kind=2, ld=64, scales=P, ld_scales=3),
                weight(kind=2, ld=63, scales=P, ld_scales=4), weight(kind=2, ld=64, ld_scales=4)):
        assert call(up=bad) == BAD
    for bad in (weight(kind=3, ld=64), weight(ld=63), weight(kind=1, ld=64),
                weight(kind=2, ld=32, scales=P, ld_scales=1)):
        assert call(down=bad) == BAD


def test_workspace_size():
    size = experts._library().experts_few_tokens_workspace_size
    n = ctypes.c_uint64(0)
    good = (10, 2, 4, 64, 96, 0)
    assert size(*good, ctypes.byref(n)) == OK and n.value >= 20 * 64 * 2
    assert size(0, *good[1:], ctypes.byref(n)) == OK and n.value == 0
    # (64 x 64 rows of 2^17 columns in two parts of two bytes: 2^31)
    assert size(64, 64, 1024, 2**17, 2**17, 0, ctypes.byref(n)) == OK and 2**31 <= n.value < 2**32
    assert size(*good, None) == BAD
    for at, value in ((1, 0), (2, 0), (3, 0), (4, 0), (5, 3), (5, -1)):
        assert size(*good[:at], value, *good[at + 1:], ctypes.byref(n)) == BAD
    for at, value in ((0, 65), (1, 65), (2, 1025), (3, 2**17 + 1), (4, 2**17 + 1)):
        assert size(*good[:at], value, *good[at + 1:], ctypes.byref(n)) == UNSUPPORTED


def test_tensors_of_the_host_are_refused():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(3, 16, 16, dtype=torch.bfloat16)
    ids, by = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        experts.few_tokens(x, w, w[:, :, :8], ids, by)

"""The 4-bit operators without a GPU: refusals, the choice of kernels, and the reference of the GPU tests
against values worked out by hand."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest
import torch

import mx4_reference
from partitioned_chip_accumulation_amd import build, experts
from test_experts_cpu import UNSUPPORTED, P, calls
from test_experts_kernels_cpu import shape
from test_experts_kernels_gpu import ROWS
from test_experts_mfma_cpu import kernels, touched_too_early
from test_experts_mx4_gpu import VIA, expected


def test_argument_errors_before_any_device_call():
    calls("experts_quantize_mx4", (P, 48, P, 3, P, 70, 10, 70, 0),
          [(0, None), (1, 47), (2, None), (3, 2), (4, None), (4, P + 1), (5, 69), (7, 0), (8, 2)])
    good = (P, 64, P, 48, P, 3, 10, P, 48, 4800, P, 3, 300, P, P, 20, 2, 4, 64, 3, 0)
    calls("experts_mx4_matmul", good,
          [(0, None), (0, P + 1), (1, 63), (2, None), (3, 47), (4, None), (5, 2), (6, 0), (7, None),
           (8, 47), (9, -1), (10, None), (11, 2), (12, -1), (13, None), (13, P + 2), (14, P + 2),
           (14, None), (16, 0), (17, 0), (18, 0), (19, 0), (20, 2)])
    lib = experts._library()
    wide = list(good)
    wide[19] = 4097  # 131104 values
    assert lib.experts_mx4_matmul(*wide, None) == UNSUPPORTED
    assert lib.experts_quantize_mx4(P, 2**20, P, 2**20, P, 2**20, 10, 2**17 + 1, 0,
                                    None) == UNSUPPORTED
    assert lib.experts_quantize_mx4(P, 48, P, 3, P, 70, 2**31, 70, 0, None) == UNSUPPORTED
    assert lib.experts_mx4_matmul(*(good[:17] + (1025,) + good[18:]), None) == UNSUPPORTED


def test_tensors_of_the_host_and_wrong_shapes_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: experts.quantize_mx4(x), lambda: experts.mx4_matmul(q, s, q, s)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("name,size,want,_", ROWS + VIA)
def test_choice_of_kernels(name, size, want, _):
    """A reduction of as many bytes leads to the same kernel as in the other products."""
    tokens, num, n, k = size
    via = (name, size, want, _) in VIA
    kernel = experts.preview("mx4_matmul", tokens, num, n, 4 * k, x_rows=tokens,
                             alignment=2 if via else 16)
    assert shape(kernel) == expected(want)


def test_every_kernel_has_a_size():
    """As far as any of many sizes finds one."""
    found = set()
    for num in (1, 2, 8, 16, 64, 300):
        for each in (1, 6, 20, 60, 100, 175, 500, 2000):
            for n in (1, 40, 136, 500, 1344, 2600, 4104, 8200):
                for k in (33, 320, 2080, 4160, 8192, 16448):
                    for alignment in (2, 16):
                        found.add(shape(experts.preview("mx4_matmul", each * num, num, n, k,
                                                        alignment=alignment)))
    assert found == {expected(c[2]) for c in ROWS + VIA}


def test_sums_of_inline_matrix_instructions_are_left_alone(tmp_path):
    """As in test_experts_mfma_cpu, which has the reason."""
    if not os.path.exists(build.hipcc()):
        pytest.skip("ROCm compiler not available")
    out = tmp_path / "device.s"
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I",
                    build.INCLUDE, "-I", build.CSRC, os.path.join(build.CSRC, "experts_mx4.hip"),
                    "-o", str(out)], check=True, capture_output=True)
    results = {name: touched_too_early(code) for name, code in kernels(out.read_text()).items()}
    assert sum(bool(count) for _, count in results.values()) == 16  # 8 kernels, two types
    assert not {name: found[:5] for name, (found, _) in results.items() if found}


def test_preview_of_the_dense_product():
    assert shape(experts.preview("mx4_matmul", 1, 0, 8192, 4096)) == (64, 64, 3, 1)
    assert shape(experts.preview("mx4_matmul", 8192, 0, 8192, 4096)) == (256, 256, 2, 1)


def test_reference_by_hand():
    x = np.zeros((1, 40))
    x[0, :9] = [4.0, 5.0, 6.0, 7.9, 0.25, 0.75, -2.5, 3.5, -0.0]
    x[0, 33] = 2.0**-130
    codes, powers = mx4_reference.quantize(x)
    # max 7.9: power 2^0. ties: 5 -> 4, 0.25 -> 0, 0.75 -> 1, -2.5 -> -2, 3.5 -> 4; 7.9 -> 6
    assert powers.tolist() == [[127, 0]]
    assert mx4_reference.values(codes, powers)[0, :9].tolist() == [4, 4, 6, 6, 0, 1, -2, 4, 0]
    # 2^-130 is an eighth of the least power: the nearest of 0 and a half is 0
    assert mx4_reference.values(codes, powers)[0, 33] == 0
    x[0, 33] = np.inf
    codes, powers = mx4_reference.quantize(x)
    assert powers.tolist() == [[127, 255]] and not codes[0, 16:].any()
    assert np.isnan(mx4_reference.values(codes, powers)[0, 32:]).all()

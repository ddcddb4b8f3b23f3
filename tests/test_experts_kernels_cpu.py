"""Which kernel a product takes: the sizes of test_experts_kernels_gpu reach the kernels that they name,
between them every kernel, and the loops over whole steps in each."""
from __future__ import annotations

import pytest

from partitioned_chip_accumulation_amd import experts, hist
from test_experts_kernels_gpu import ROWS, VIA, WEIGHTS

STEP = 128  # bytes of reduction


def shape(kernel):
    return kernel.rows, kernel.cols, kernel.stages, kernel.direct


def runs_whole_steps(kernel, steps):
    """The loop without checks starts where a step and what it fetches ahead lie before the end: two
    steps ahead of their use through registers, as many as there are stages straight to LDS."""
    ahead = kernel.stages if kernel.direct else 4
    return steps > ahead + max(kernel.stages, 2) - 1


@pytest.mark.parametrize("name,size,want,want_dx", ROWS + VIA)
def test_rows(name, size, want, want_dx):
    tokens, num, n, k = size
    via = (name, size, want, want_dx) in VIA
    kernels = {
        "matmul": experts.preview("matmul", tokens, num, n, k, x_rows=tokens,
                                  alignment=2 if via else 16),
        # rows of quantised operands start at multiples of 16 bytes, the weights' do not
        "int8": experts.preview("int8_matmul", tokens, num, n, 2 * k + via, x_rows=tokens),
        "dx": experts.preview("matmul_dx", tokens, num, k, n),
    }
    for product, kernel in kernels.items():
        expected = want_dx or want if product == "dx" else want
        if product == "dx" and want[2] == 0:
            expected = (32, 128, 3, 1) if n % 8 == 0 else (32, 128, 2, 0)
        assert shape(kernel) == expected, product
        if kernel.stages and "short" not in name:
            assert runs_whole_steps(kernel, 2 * k // STEP), product


@pytest.mark.parametrize("name,size,want", WEIGHTS)
def test_weights(name, size, want):
    tokens, num, n, k = size
    kernel = experts.preview("matmul_dw", tokens, num, n, k, x_rows=tokens)
    assert shape(kernel) == want
    if num <= 3:  # (rows of several times 64 for an expert)
        assert runs_whole_steps(kernel, tokens // num // 2 // 64)


def test_every_kernel_has_a_size():
    """As far as any of many sizes finds one."""
    found = {"matmul": set(), "int8_matmul": set(), "matmul_dx": set(), "matmul_dw": set()}
    widths = (1, 40, 128, 136, 500, 1344, 2600, 4104, 8200, 33)
    for product, kernels in found.items():
        for num in (1, 2, 8, 16, 64, 300):
            for each in (1, 6, 20, 60, 100, 175, 500, 2000):
                for n in widths:
                    for k in (33, 80, 528, 1040, 2048, 4112):
                        kernels.add(shape(experts.preview(product, each * num, num, n, k)))
    tested = {c[2] for c in ROWS + VIA}
    assert found["matmul"] == tested and found["int8_matmul"] == tested
    of_dx = {(c[3] or c[2]) for c in ROWS + VIA if c[2][2]}
    assert found["matmul_dx"] == of_dx
    assert found["matmul_dw"] == {c[2] for c in WEIGHTS}


def test_preview_follows_the_operands():
    def of(**change):
        return shape(experts.preview("matmul", 32768, 16, 4096, 4096, **change))

    assert of() == of(x_rows=8192) == (256, 256, 2, 1)
    # addresses or rows off 16 bytes, and rows past 32-bit offsets, pass through registers
    assert of(alignment=2) == of(lda=4100) == of(ldb=4097) == (256, 128, 2, 0)
    assert of(lda=2**24) == of(x_rows=2**20, lda=4096) == (256, 128, 2, 0)
    assert shape(experts.preview("int8_matmul", 1, 0, 8192, 4096)) == (16, 16, 0, 0)


@pytest.mark.parametrize("product,sizes,change", [
    ("matmul", (0, 4, 64, 64), {}), ("matmul", (8, 0, 64, 64), {}), ("matmul", (8, 4, 0, 64), {}),
    ("matmul", (8, 4, 64, 64), {"lda": 63}), ("matmul_dx", (8, 4, 64, 32), {"lda": 63}),
    ("matmul", (8, 4, 64, 64), {"ldb": 63}), ("matmul", (8, 4, 64, 64), {"alignment": 3}),
    ("matmul", (8, 4, 64, 64), {"alignment": 0}), ("matmul_dx", (8, 4, 64, 64), {"x_rows": 4}),
    ("int8_matmul", (8, 0, 64, 64), {"x_rows": 4})])
def test_preview_refuses(product, sizes, change):
    with pytest.raises(hist.HistError):
        experts.preview(product, *sizes, **change)

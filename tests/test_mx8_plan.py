"""Which kernel a product of MX8 with MX4 takes, without a GPU: the shapes that the GPU
tests multiply take every kernel that any shape takes."""
import ctypes
import math
import random

import pytest

from lossless_bit_weight_amd import mx8
from tests.mx8_cases import KERNEL_SHAPES


def _kernel(shape):
    name, slices = mx8.mx8_gemm_plan(*shape)
    return name, slices > 1


@pytest.mark.parametrize("kernel", list(KERNEL_SHAPES), ids=str)
def test_shapes_take_their_kernel(kernel):
    for shape in KERNEL_SHAPES[kernel]:
        assert _kernel(shape) == kernel, shape


def test_no_shape_takes_another():
    rng = random.Random(7)

    def size(most):
        return int(round(math.exp(rng.uniform(0, math.log(most)))))

    found = {_kernel((size(8192), size(150000), 32 * size(2048))) for _ in range(60000)}
    # large ones and limits
    found |= {_kernel(s) for s in ((1 << 24, 1, 32), (1 << 24, 8192, 5120), (1, 1 << 27, 32),
                                   (1, 16, (1 << 24) - 32), (4096, 34816, 17408))}
    assert found == set(KERNEL_SHAPES)


def test_slices_are_those_of_the_workspace():
    for shapes in KERNEL_SHAPES.values():
        for M, N, K in shapes:
            slices = mx8.mx8_gemm_plan(M, N, K)[1]
            need = slices * M * ((N + 3) // 4 * 4) * 4 if slices > 1 else 0
            assert mx8.mx8_gemm_workspace_bytes(M, N, K) == need


@pytest.mark.parametrize("shape", [(0, 16, 32), (-1, 16, 32), (1, 0, 32), (1, 16, 33),
                                   ((1 << 24) + 1, 1, 32), (1, (1 << 27) + 1, 32)])
def test_refused_shapes_have_no_kernel(shape):
    n = ctypes.c_int(7)
    assert mx8.lib().mx8_gemm_plan(*shape, ctypes.byref(n)) is None and n.value == 0
    assert mx8.lib().mx8_gemm_plan(*shape, None) is None
    with pytest.raises(mx8.MX8Error):
        mx8.mx8_gemm_plan(*shape)

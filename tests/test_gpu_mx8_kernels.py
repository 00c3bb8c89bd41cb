"""Products of MX8 with MX4 through every kernel by its own rule (tests/test_mx8_plan.py
holds that the shapes take them), exact."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4, mx8
from tests.gpu_util import require_gpu
from tests.mx8_cases import SHAPES

pytestmark = pytest.mark.gpu

OUT = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _exact(x, w):
    """Both outputs of the product of x and w (fp32, on the GPU, held by MX8 and MX4 as they
    are) are those of the 64-bit product, rounded to their type."""
    xq, wq = mx8.mx8_quantize(x), mx4.mx4_quantize(w)
    assert torch.equal(mx8.mx8_dequantize(xq, torch.float32), x)
    assert torch.equal(mx4.mx4_dequantize(wq, torch.float32), w)
    want = x.double() @ w.double().T
    for out in OUT:
        assert torch.equal(mx8.mx8_gemm(xq, wq, out), want.to(out)), out


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers(M, N, K):
    """Sums of at most 84 K, below 2^22 for the longest K: fp32 holds every partial sum."""
    rng = np.random.default_rng(M + N + K)
    x = rng.integers(-14, 15, (M, K)).astype(np.float32)
    w = rng.choice([0.0, 1.0, 2.0, 3.0, -4.0, 6.0, -1.0], (N, K)).astype(np.float32)
    w[:, ::32] = 4.0                            # the scale of every block is 1
    _exact(torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda())

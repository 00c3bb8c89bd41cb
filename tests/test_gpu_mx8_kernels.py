"""Products of MX8 with MX4 through every kernel by its own rule (tests/test_mx8_plan.py
holds that the shapes take them), exact."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4, mx8
from tests.gpu_util import require_gpu
from tests.mx8_cases import SHAPES, edges

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


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_as_far_apart_as_they_go(M, N, K):
    """+-448 times 6 beside 1/4 times 1/2 in the same eights: 13 bits, none of them lost."""
    x, w = (torch.from_numpy(v).float().cuda() for v in edges(M, N, K))
    # of magnitudes in any order: multiples of 1/8, below fp32's 24 bits of them
    assert float((x.abs() @ w.abs().T).max()) < 2.0 ** 21 * (1 - 2.0 ** -10)
    _exact(x, w)


@pytest.mark.parametrize("big,six", [(448.0, 6.0), (256.0, 4.0), (288.0, 6.0)])
def test_every_pair_of_places_in_a_block(big, six):
    """One product of each kind alone in a block, in every two places of it."""
    x, w = torch.zeros(32 * 32, 32), torch.zeros(32 * 32, 32)
    for i in range(32):
        for j in range(32):
            if i != j:
                x[32 * i + j, i], x[32 * i + j, j] = big, -0.25
                w[32 * i + j, i], w[32 * i + j, j] = six, 0.5
    x, w = x.cuda(), w.cuda()
    _exact(x, w)


# 256 * 4 beside what fine steps hold: 13 bits below it is kept, 14 is lost in its own eight
# and kept in another
@pytest.mark.parametrize("small,kept", [(0.25, True), (0.125, False), (2.0 ** -6, False),
                                        (2.0 ** -9, False)])
def test_what_fine_steps_lose(small, kept):
    x, w = torch.zeros(32 * 32, 64), torch.zeros(32 * 32, 64)
    want = torch.full((32 * 32,), 1024.0)
    for i in range(32):
        for j in range(32):
            r = 32 * i + j
            x[r, i], w[r, i] = 256.0, 4.0
            if i != j:
                x[r, j], w[r, j] = small, 0.5
                if kept or i // 8 != j // 8:
                    want[r] += small / 2
    xq = mx8.mx8_quantize(x.cuda(), fine=True)
    assert torch.equal(mx8.mx8_dequantize(xq, torch.float32), x.cuda())
    got = mx8.mx8_gemm(xq, mx4.mx4_quantize(w.cuda())).diagonal().cpu()
    assert torch.equal(got, want)

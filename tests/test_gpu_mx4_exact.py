"""MX4 operators on the GPU where the true result is a number that fp32 holds:
every sum is one of whole numbers below 2^24 (times one power of two), so the
kernels have to return it exactly, rounded once to the output type."""
import numpy as np
import pytest
import torch

from lossless_bit_weight_amd import mx4
from tests import mx4_ref as ref
from tests.gpu_util import require_gpu
from tests.test_gpu_mx4 import GEMM_KERNELS, GEMM_SHAPES

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _dev(v, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(v).astype(np.float32)).cuda().to(dtype)


def _assert_equal(y, want, out):
    """y is `want` (exact in fp32) in its type."""
    if out == "bf16":
        want = ref.bf16_to_f64(ref.f64_to_bf16_bits(want))
    got = y.float().cpu().numpy().astype(np.float64)
    bad = np.argwhere(got != want)
    assert bad.size == 0, "%d of %d differ, the first at %s: %r, not %r" % (
        len(bad), want.size, bad[0], got[tuple(bad[0])], want[tuple(bad[0])])


# ---- hidden values of the expert layer ------------------------------------------------

# one token; four of few experts (slots of one kernel); slots of up to 4 and of up to 16
# rows; a long I; many workgroups of the down product
HIDDEN_SHAPES = [(1, 64, 96, 1), (1, 160, 1056, 9), (4, 1024, 2048, 1), (7, 96, 160, 3),
                 (40, 64, 96, 24), (40, 96, 4128, 2), (90, 96, 4128, 40), (128, 1056, 64, 64)]


def _hidden_case(T, H, I, E, seed):
    """x, gate and up weights whose hidden values are whole numbers of up to 23 bits:
    g = sum of digit * 8^k, 585 and more (so exp(-g) = 0 and silu(g) = g), u alike."""
    rng = np.random.default_rng(seed)
    w13 = rng.choice([0.0, 1.0, 2.0, -3.0], (E, 2 * I, H))
    w13[:, :I, :4] = rng.choice([1.0, 2.0, 3.0, 4.0, 6.0], (E, I, 4))
    w13[:, I:, :4] = rng.choice([1.0, 2.0, 3.0], (E, I, 4))
    assert np.array_equal(ref.rounded(w13), w13)
    x = np.zeros((T, H))
    for t in range(T):
        x[t, :4] = 8.0 ** rng.permutation(4)
    expert = rng.integers(0, E, T)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[np.arange(T), expert] = 9.0
    gu = np.matmul(x[:, None, :], w13[expert].transpose(0, 2, 1))[:, 0]
    h = gu[:, :I] * gu[:, I:]
    assert gu[:, :I].min() >= 585 and 0 < h.min() and h.max() < 1 << 23
    return rng, x, logits, expert, w13, h


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I,E", HIDDEN_SHAPES)
def test_hidden_values_keep_24_bits(T, H, I, E, out):
    """One expert a token (its share is 1) whose down rows subtract two hidden values
    that lie next to each other in size: small differences of numbers of 23 bits."""
    rng, x, logits, expert, w13, h = _hidden_case(T, H, I, E, 7 * T + I)
    w2 = np.zeros((E, H, I))
    for e in range(E):
        near = np.argsort(h[np.argmax(expert == e)], kind="stable")
        a = rng.integers(0, I - 1, H)
        w2[e, np.arange(H), near[a + 1]] = 1.0
        w2[e, np.arange(H), near[a]] = -1.0
        w2[e, ::7] = 0.0
        w2[e, np.arange(0, H, 7), rng.integers(0, I, len(range(0, H, 7)))] = -1.0    # h itself
    assert np.array_equal(ref.rounded(w2), w2)
    want = np.matmul(w2[expert], h[:, :, None])[:, :, 0]
    y = mx4.mx4_moe(_dev(x), torch.from_numpy(logits).cuda(), mx4.mx4_quantize(_dev(w13)),
                    mx4.mx4_quantize(_dev(w2)), 1, out_dtype=TYPES[out])
    _assert_equal(y, want, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I,E", [(1, 64, 96, 2), (40, 64, 96, 24), (40, 96, 1056, 2)])
def test_hidden_values_at_the_top_of_fp32(T, H, I, E, out):
    """Hidden values within 2^-9 of the largest fp32 number, which no BF16 holds: finite,
    so their products with small weights are too."""
    digits = np.array(np.meshgrid(*[[1, 2, 3, 4, 6]] * 4)).reshape(4, -1).T
    value = digits @ 8 ** np.arange(4)
    product = np.outer(value, value)
    pairs = np.argwhere((product >= (1 << 22) - (1 << 13)) & (product < 1 << 22))
    rng = np.random.default_rng(T)
    pick = pairs[rng.integers(0, len(pairs), (E, I))]
    w13 = np.zeros((E, 2 * I, H))
    sign = rng.choice([-1.0, 1.0], (E, I))
    w13[:, :I, :4], w13[:, I:, :4] = digits[pick[..., 0]], sign[..., None] * digits[pick[..., 1]]
    x = np.zeros((T, H))
    x[:, :4] = 8.0 ** np.arange(4) * 2.0 ** 53
    w2 = np.zeros((E, H, I))
    at = rng.integers(0, I, (E, H))
    np.put_along_axis(w2, at[..., None], 2.0 ** -100, axis=2)
    for w in (w13, w2):
        assert np.array_equal(ref.rounded(w), w)
    expert = rng.integers(0, E, T)
    logits = np.zeros((T, E), np.float32)
    logits[np.arange(T), expert] = 9.0
    h = sign * product[pick[..., 0], pick[..., 1]] * 2.0 ** 106
    assert np.abs(h).max() <= np.finfo(np.float32).max
    want = (np.take_along_axis(h, at, 1) * 2.0 ** -100)[expert]
    y = mx4.mx4_moe(_dev(x), torch.from_numpy(logits).cuda(), mx4.mx4_quantize(_dev(w13)),
                    mx4.mx4_quantize(_dev(w2)), 1, out_dtype=TYPES[out])
    _assert_equal(y, want, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,I,E", [(1, 96, 2), (40, 96, 24), (40, 1056, 2)])
def test_infinite_hidden_value(T, I, E, out):
    """g u past fp32's range: its products are infinite, with the weight's sign."""
    H = 64
    w13 = np.zeros((E, 2 * I, H))
    w13[:, 5, 0] = w13[:, I + 5, 0] = 4.0
    x = np.zeros((T, H))
    x[:, 0] = 2.0 ** 70
    w2 = np.random.default_rng(T).choice([-2.0, 1.0], (E, H, I))
    expert = np.arange(T) % E
    logits = np.zeros((T, E), np.float32)
    logits[np.arange(T), expert] = 9.0
    y = mx4.mx4_moe(_dev(x), torch.from_numpy(logits).cuda(), mx4.mx4_quantize(_dev(w13)),
                    mx4.mx4_quantize(_dev(w2)), 1, out_dtype=TYPES[out])
    assert np.array_equal(y.float().cpu().numpy(), w2[expert][:, :, 5] * np.inf)


# ---- products ------------------------------------------------------------------------

def _whole(shape, seed):
    """Whole numbers from -2 to 2: MX4 holds them, and a sum of fewer than 2^22 products
    of two is exact in fp32 in any order."""
    return np.random.default_rng(seed).integers(-2, 3, shape).astype(np.float64)


# past the lengths that one slice, one wave or one unit of a kernel takes
LONG = [(M, N, 65536) for M in (1, 3, 11, 16) for N in (70, 2600)] + [
    (27, 300, 65536), (40, 300, 65536), (64, 2600, 65536), (100, 300, 65536), (200, 520, 65536),
    (2, 16400, 20000), (13, 16400, 20000), (27, 16400, 20000), (50, 16400, 20000),
    (300, 1000, 20000)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES + GEMM_KERNELS + LONG)
def test_products_of_whole_numbers(M, N, K):
    """Every kernel, every cut of K: no group of K may be left out, taken twice or met by
    another one's scale."""
    K -= K % 32
    x, w = _whole((M, K), M + K), _whole((N, K), N + K + 1)
    for k in range(0, K, 32):                  # scales of their own for every block of K
        s = 2.0 ** (k // 32 % 3)
        x[:, k:k + 32] *= s
        w[:, k:k + 32] /= s
    want = (torch.from_numpy(x).cuda() @ torch.from_numpy(w).cuda().T).cpu().numpy()
    xd, wq = _dev(x), mx4.mx4_quantize(_dev(w))
    for a in (xd, mx4.mx4_quantize(xd)):
        for out in TYPES:
            _assert_equal(mx4.mx4_gemm(a, wq, out_dtype=TYPES[out]), want, out)

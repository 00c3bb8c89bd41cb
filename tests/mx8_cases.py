"""Shapes that take every kernel of the product of MX8 with MX4, whole and in slices of
K, most of them with ragged rows, columns and last groups; and operands at the edge of
what the matrix units add without loss."""
from __future__ import annotations

import numpy as np

# (kernel, in slices): shapes
KERNEL_SHAPES = {
    ("small_kernel<1, 4>", False): [(1, 1, 32), (4, 500, 2336), (37, 65, 1056)],
    ("small_kernel<1, 8>", False): [(3, 77, 5120), (5, 23, 2144)],
    ("small_kernel<2, 4>", False): [(9, 16400, 1056), (12, 20001, 3584), (16, 65530, 544),
                                    (9, 26417, 2336)],
    ("mid_kernel<1, 4, 1, 1>", False): [(2, 21231, 3840), (15, 24005, 4128)],
    ("mid_kernel<1, 5, 1, 1>", False): [(1, 16623, 3840), (16, 16500, 4192)],
    ("mid_kernel<1, 2, 2, 2>", False): [(18, 2098, 1088), (5, 4292, 2208), (1183, 1, 8480)],
    ("mid_kernel<1, 2, 2, 2>", True): [(15, 31, 8480), (10, 501, 17376)],
    ("mid_kernel<1, 4, 2, 2>", False): [(2245, 51, 1088), (61, 3999, 1120)],
    ("mid_kernel<1, 4, 2, 2>", True): [(186, 34, 12192), (17, 410, 9760)],
    ("mid_kernel<2, 4, 2, 1>", False): [(3273, 67, 1600)],
    ("mid_kernel<2, 4, 2, 1>", True): [(600, 33, 18656), (17, 1243, 19424)],
    ("tile_kernel<2, 2, 4, 2>", False): [(2884, 116, 32), (18, 16999, 1056)],
    ("tile_kernel<2, 2, 4, 2>", True): [(70, 1030, 17408), (130, 520, 17408), (96, 1444, 21088),
                                        (1443, 4, 16480)],
    ("tile_kernel<4, 2, 4, 2>", False): [(2734, 1814, 32)],
    ("tile_kernel<4, 2, 4, 2>", True): [(33, 5003, 17376), (2623, 1, 29696)],
    ("tile_kernel<4, 2, 5, 2>", False): [(1789, 2830, 32)],
    ("tile_kernel<4, 2, 5, 2>", True): [(936, 140, 16704), (1146, 132, 10816)],
    ("tile_kernel<4, 4, 4, 1>", False): [(1609, 6281, 32), (700, 17001, 544)],
    ("tile_kernel<4, 4, 4, 1>", True): [(66, 11052, 9568)],
}
SHAPES = [s for shapes in KERNEL_SHAPES.values() for s in shapes]


def edges(M: int, N: int, K: int) -> tuple:
    """(x [M, K], w [N, K]) whose products lie as far apart as MX8 and MX4 let them under
    scales of 1: in each block of x one or two of +-448, the second of the other sign in the
    same eight, among multiples of 1/4; in each of w +-6 among +-0.5 and others.  Every sum
    of products is a multiple of 1/8 below 2^21, which fp32 holds."""
    rng = np.random.default_rng(M + N + K)
    n = K // 32
    x = rng.choice([0.25, -0.25, 0.75, -0.25, 0.5, 1.75, 0.0], (M, n, 32))
    at, sign = rng.integers(0, 32, (M, n)), rng.choice([-448.0, 448.0], (M, n))
    np.put_along_axis(x, at[..., None], sign[..., None], 2)
    beside = at ^ rng.integers(1, 8, (M, n))
    two = rng.random((M, n)) < 0.5
    np.put_along_axis(x, np.where(two, beside, at)[..., None],
                      np.where(two, -sign, sign)[..., None], 2)
    w = rng.choice([0.5, -0.5, 0.5, 1.5, -6.0, 6.0, 0.0], (N, n, 32))
    np.put_along_axis(w, rng.integers(0, 32, (N, n))[..., None],
                      rng.choice([-6.0, 6.0], (N, n))[..., None], 2)
    return x.reshape(M, K), w.reshape(N, K)


def summed_in_eights(x: np.ndarray, w: np.ndarray, bits: int) -> np.ndarray:
    """x w^T where each eight neighbours along K lose what lies more than `bits` below the
    exponent (of the operands, added) of their largest product."""
    y = np.zeros((len(x), len(w)))
    with np.errstate(divide="ignore"):
        ex, ew = (np.floor(np.log2(np.abs(v))) for v in (x, w))
    for k in range(0, x.shape[1], 8):
        p = x[:, None, k:k + 8] * w[None, :, k:k + 8]
        e = (ex[:, None, k:k + 8] + ew[None, :, k:k + 8]).max(-1, keepdims=True)
        step = np.exp2(np.where(np.isfinite(e), e, 0.0) - bits)
        y += (np.trunc(p / step) * step).sum(-1)
    return y

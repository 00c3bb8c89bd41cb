"""Shapes that take every kernel of the product of MX8 with MX4, whole and in slices of
K, most of them with ragged rows, columns and last groups."""
from __future__ import annotations

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
